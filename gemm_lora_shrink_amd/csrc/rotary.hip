// Rotary positions, the norm of each head before them, and the tokens' rows
// of the paged cache, in one pass over the q/k/v rows.
//
// A pair (a, b) of a head turns by the angle of its frequency and the token's
// position: a' = a c - b s, b' = b c + a s.  With the norm, x[i] is first
// multiplied by w[i] / sqrt(mean(x^2) + eps).  Everything is fp32 between one
// load and one store of each element.
//
// The pass moves 2 (q_heads + 2 kv_heads) d elements a token and computes next
// to nothing, so it is bound by memory, or for a decode batch by its chain of
// loads: the token's position, then its row of the table.  The x loads do not
// wait for that chain.  Measured: 8192 tokens of 32 + 2 x 8 bf16 heads of 128 with
// norms 43.5 us (201 MB, 4.6 TB/s, a large copy's rate); 4097 tokens of 16 + 2 x 16
// fp16 heads of 256, 64 elements rotated, 42.7 us (201 MB); 64 tokens of 32 + 2 x 8
// 11 us, the time of the call on the host.
#include <cmath>

#include "attention.h"

namespace lora {

namespace {

constexpr int kThreads = 256;

// ---- the table ------------------------------------------------------------

struct TableParams {
  float* table;
  int64_t first, n;
  double magnitude;
  int32_t half, run;  // positions of a thread
  FastDiv by_half;
  double turns[LORA_MAX_HEAD_DIM / 2];  // frequency / (2 pi)
  double step[LORA_MAX_HEAD_DIM];       // cosine and sine of the frequency
};

// A thread fills `run` positions of one pair.  At the first, the position times
// the frequency, in turns, is reduced to its fraction in 64 bits before cosine
// and sine, so that a far position loses nothing but the product's own rounding
// (2^-53 of the turns); from there on a position turns the one before it by the
// frequency, in 64 bits too: four products in place of a cosine and a sine, for
// 2^-52 more a step, far below the table's own 2^-24.
// With a cosine, a sine and a 64-bit division at every position the kernel was
// bound by those: 29.0 us for 131072 positions of 64 pairs (67 MB), now 12.1 (5.5 TB/s).
__global__ __launch_bounds__(kThreads) void rope_table_kernel(TableParams p) {
  const uint32_t e = blockIdx.x * kThreads + threadIdx.x, r = p.by_half.div(e);
  const int i = (int)(e - r * p.by_half.d);
  const int64_t pos = (int64_t)r * p.run;
  const int n = (int)(p.n - pos < p.run ? p.n - pos : p.run);
  if (n <= 0) return;
  const double turns = (double)(p.first + pos) * p.turns[i], dc = p.step[2 * i], ds = p.step[2 * i + 1];
  double s, c;
  sincospi(2.0 * (turns - rint(turns)), &s, &c);
  s *= p.magnitude;
  c *= p.magnitude;
  float* row = p.table + pos * 2 * p.half + i;
#pragma unroll 4
  for (int j = 0; j < n; ++j) {
    row[0] = (float)c;
    row[p.half] = (float)s;
    row += 2 * p.half;
    const double next = c * dc - s * ds;
    s = s * dc + c * ds;
    c = next;
  }
}

// ---- the rotation -----------------------------------------------------------

// Eight consecutive elements, as loaded and as fp32.
template <typename Elem> struct Eight {
  static constexpr int kWords = sizeof(Elem) / 2;  // 16-byte pieces
  u32x4 raw[kWords];
  __device__ inline void load(const Elem* p, bool ok) {
#pragma unroll
    for (int w = 0; w < kWords; ++w) raw[w] = ld16_or0(reinterpret_cast<const u32x4*>(p) + w, ok);
  }
  __device__ inline void to_float(float* f) const {
#pragma unroll
    for (int w = 0; w < kWords; ++w) Traits<Elem>::to_float(raw[w], f + w * Traits<Elem>::kVec);
  }
  __device__ inline void store(Elem* p) const {
#pragma unroll
    for (int w = 0; w < kWords; ++w) reinterpret_cast<u32x4*>(p)[w] = raw[w];
  }
};
template <typename Elem> __device__ inline Eight<Elem> rounded(const float* f) {
  Eight<Elem> e;
  if constexpr (sizeof(Elem) == 4) {
#pragma unroll
    for (int w = 0; w < 2; ++w)
      e.raw[w] = u32x4{__float_as_uint(f[4 * w]), __float_as_uint(f[4 * w + 1]), __float_as_uint(f[4 * w + 2]),
                       __float_as_uint(f[4 * w + 3])};
  } else if constexpr (Traits<Elem>::kDtype == LORA_BF16) {
    e.raw[0] = u32x4{pack2_bf16(f[0], f[1]), pack2_bf16(f[2], f[3]), pack2_bf16(f[4], f[5]), pack2_bf16(f[6], f[7])};
  } else {
    e.raw[0] = u32x4{pack2_f16(f[0], f[1]), pack2_f16(f[2], f[3]), pack2_f16(f[4], f[5]), pack2_f16(f[6], f[7])};
  }
  return e;
}
template <typename Elem> __device__ inline Elem one_rounded(float f) { return static_cast<Elem>(f); }

// Where head h of token t comes from and its place in the out rows (null: none).
template <typename Elem> struct HeadPtrs {
  const Elem* in;
  Elem* out;
  bool turns;  // a q or k head
};
template <typename Elem>
__device__ inline HeadPtrs<Elem> head_ptrs(const RotaryParams& p, int64_t t, int h) {
  HeadPtrs<Elem> r;
  const int kv = h < p.hq ? 0 : (h < p.hq + p.hk ? h - p.hq : h - p.hq - p.hk);
  r.turns = h < p.hq + p.hk;
  if (h < p.hq) {
    r.in = static_cast<const Elem*>(p.q) + t * p.ldq + (int64_t)h * p.d;
    r.out = static_cast<Elem*>(p.q_out) + t * p.ldqo + (int64_t)h * p.d;
  } else if (r.turns) {
    r.in = static_cast<const Elem*>(p.k) + t * p.ldk + (int64_t)kv * p.d;
    r.out = p.k_out ? static_cast<Elem*>(p.k_out) + t * p.ldko + (int64_t)kv * p.d : nullptr;
  } else {
    r.in = static_cast<const Elem*>(p.v) + t * p.ldv + (int64_t)kv * p.d;
    r.out = nullptr;
  }
  return r;
}
template <typename Elem>
__device__ inline Elem* cache_ptr(const RotaryParams& p, int row, int h) {
  if (!p.cache.k || h < p.hq || row < 0 || row >= p.n_rows) return nullptr;
  const int64_t page = p.cache.page.div((uint32_t)row), place = row - page * p.cache.page.d;
  return h < p.hq + p.hk ? static_cast<Elem*>(p.cache.k) + page * p.cache.k_page + (h - p.hq) * p.cache.k_head +
                               place * p.cache.k_row
                         : static_cast<Elem*>(p.cache.v) + page * p.cache.v_page +
                               (h - p.hq - p.hk) * p.cache.v_head + place * p.cache.v_row;
}

// Whole 16-byte pieces: d and rot multiples of 16.  A head is d / 16 units of
// two 8-element chunks, one lane each; the first rot / 16 units turn: HALF
// pairs chunk u with chunk u + rot / 16, INTERLEAVED takes chunks 2u and
// 2u + 1.  A lane group (a power of two, for the norm's sum over the head)
// walks HPG heads of one token, which share the lane's cosines and sines; the
// groups of a token take adjacent heads at each step, so a wave reads
// contiguous memory.
template <typename Elem, int HPG, bool NORM, bool HALF>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryParams p) {
  warm_args(p);
  const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int u = (int)(g & ((1 << p.lane_shift) - 1));
  const int64_t rest = g >> p.lane_shift;
  const int64_t t = p.groups.div((uint32_t)rest);
  if (t >= p.T) return;  // the same for a whole lane group
  const int grp = (int)(rest - t * p.groups.d);
  const int heads = p.hq + p.hk + (p.cache.k ? p.hk : 0);
  const bool there = u < p.units;
  const int turning = p.rot / 16;
  const bool turn = u < turning;
  const int c0 = HALF ? (turn ? u : 2 * u) : 2 * u;
  const int c1 = HALF && turn ? u + turning : c0 + 1;

  const int pos = p.positions[t];
  const int row = p.cache.k ? p.cache_rows[t] : -1;
  HeadPtrs<Elem> ptr[HPG];
  Eight<Elem> x[HPG][2];
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = grp + i * p.groups.d;
    const bool ok = there && h < heads;
    ptr[i] = head_ptrs<Elem>(p, t, h < heads ? h : 0);
    x[i][0].load(ptr[i].in + 8 * c0, ok);
    x[i][1].load(ptr[i].in + 8 * c1, ok);
  }
  const bool known = pos >= 0 && pos < p.n_positions;
  float c[8], s[8];
  const float* at = p.table + (int64_t)(known ? pos : 0) * p.rot + 8 * u;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const f32x4 cw = ldf4_or0(at + 4 * w, turn), sw = ldf4_or0(at + p.rot / 2 + 4 * w, turn);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[4 * w + j] = cw[j];
      s[4 * w + j] = sw[j];
    }
  }
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    const int h = grp + i * p.groups.d;
    const bool ok = there && h < heads;
    Eight<Elem> y0 = x[i][0], y1 = x[i][1];
    float f[16];
    if constexpr (NORM) {
      const void* wv = h < p.hq ? p.qw : p.kw;
      Eight<Elem> w0, w1;
      const Elem* wp = static_cast<const Elem*>(wv);
      const bool weighed = ok && wv && h < p.hq + p.hk;
      w0.load(wp + 8 * c0, weighed);
      w1.load(wp + 8 * c1, weighed);
      y0.to_float(f);
      y1.to_float(f + 8);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) ss = __builtin_fmaf(f[j], f[j], ss);
      for (int o = 1 << p.lane_shift >> 1; o; o >>= 1) ss += __shfl_xor(ss, o);
      const float r = 1.0f / sqrtf(ss / (float)p.d + p.eps);
      float w[16];
      w0.to_float(w);
      w1.to_float(w + 8);
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = f[j] * r * (wv ? w[j] : 1.0f);
    } else {
      y0.to_float(f);
      y1.to_float(f + 8);
    }
    if (!ok || !known) continue;
    if (ptr[i].turns) {
      if (turn) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ia = HALF ? j : 2 * j, ib = HALF ? j + 8 : 2 * j + 1;
          const float a = f[ia], b = f[ib];
          f[ia] = a * c[j] - b * s[j];
          f[ib] = b * c[j] + a * s[j];
        }
      }
      if (NORM || turn) {
        y0 = rounded<Elem>(f);
        y1 = rounded<Elem>(f + 8);
      }
    }
    Elem* cache = cache_ptr<Elem>(p, row, h);
    if (ptr[i].out) {
      y0.store(ptr[i].out + 8 * c0);
      y1.store(ptr[i].out + 8 * c1);
    }
    if (cache) {
      y0.store(cache + 8 * c0);
      y1.store(cache + 8 * c1);
    }
  }
}

// Any even rot and any d: 16 lanes a head, a lane takes every 16th pair of the
// rotated part and then of the rest, element by element.  A lane holds both
// elements of a pair before it stores them, and the norm's sum is complete
// before any store, so this works in place too.
template <typename Elem, bool NORM>
__global__ __launch_bounds__(kThreads) void rotary_pairs_kernel(RotaryParams p) {
  warm_args(p);
  const int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int lane = (int)(g & 15);
  const int64_t rest = g >> 4;
  const int64_t t = p.groups.div((uint32_t)rest);
  if (t >= p.T) return;
  const int h = (int)(rest - t * p.groups.d);  // one head a group
  const HeadPtrs<Elem> ptr = head_ptrs<Elem>(p, t, h);
  Elem* cache = cache_ptr<Elem>(p, p.cache.k ? p.cache_rows[t] : -1, h);
  const int pos = p.positions[t];
  float r = 1.0f;
  const Elem* w = nullptr;
  if (NORM && ptr.turns) {
    float ss = 0.f;
    for (int e = lane; e < p.d; e += 16) {
      const float x = (float)ptr.in[e];
      ss = __builtin_fmaf(x, x, ss);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor(ss, o);
    r = 1.0f / sqrtf(ss / (float)p.d + p.eps);
    w = static_cast<const Elem*>(h < p.hq ? p.qw : p.kw);
  }
  if (pos < 0 || pos >= p.n_positions) return;
  const float* at = p.table + (int64_t)pos * p.rot;
  const int half = p.rot / 2;
  for (int j = lane; j < p.d / 2; j += 16) {
    const bool turn = j < half && ptr.turns;
    const int e0 = j < half && p.layout == LORA_ROPE_HALF ? j : 2 * j;
    const int e1 = j < half && p.layout == LORA_ROPE_HALF ? j + half : 2 * j + 1;
    Elem y0 = ptr.in[e0], y1 = ptr.in[e1];
    if (ptr.turns && (NORM || turn)) {
      float a = (float)y0, b = (float)y1;
      if (NORM) {
        a = a * r * (w ? (float)w[e0] : 1.0f);
        b = b * r * (w ? (float)w[e1] : 1.0f);
      }
      const float c = turn ? at[j] : 1.0f, s = turn ? at[half + j] : 0.0f;
      y0 = one_rounded<Elem>(turn ? a * c - b * s : a);
      y1 = one_rounded<Elem>(turn ? b * c + a * s : b);
    }
    if (ptr.out) {
      ptr.out[e0] = y0;
      ptr.out[e1] = y1;
    }
    if (cache) {
      cache[e0] = y0;
      cache[e1] = y1;
    }
  }
}

template <typename Elem, int HPG>
void launch_units(const RotaryParams& p, unsigned blocks, hipStream_t stream) {
  const bool half = p.layout == LORA_ROPE_HALF;
  const dim3 g(blocks), b(kThreads);
  if (p.norm && half) hipLaunchKernelGGL((rotary_kernel<Elem, HPG, true, true>), g, b, 0, stream, p);
  else if (p.norm) hipLaunchKernelGGL((rotary_kernel<Elem, HPG, true, false>), g, b, 0, stream, p);
  else if (half) hipLaunchKernelGGL((rotary_kernel<Elem, HPG, false, true>), g, b, 0, stream, p);
  else hipLaunchKernelGGL((rotary_kernel<Elem, HPG, false, false>), g, b, 0, stream, p);
}

// How a call's heads (q, k and v) are laid over threads.
struct RotaryPlan {
  bool pieces;  // 16-byte pieces
  int lane_shift, heads_of_group, groups;
  int64_t threads;
};
RotaryPlan rotary_plan(int32_t T, int heads, int32_t d, int32_t rot) {
  RotaryPlan a{};
  a.pieces = d % 16 == 0 && rot % 16 == 0;
  a.heads_of_group = 1;
  a.lane_shift = 4;
  if (a.pieces) {
    a.lane_shift = 0;
    while ((16 << a.lane_shift) < d) ++a.lane_shift;
    const int64_t lanes = ((int64_t)T * heads) << a.lane_shift;
    if (lanes >= (int64_t)kThreads * 4096) a.heads_of_group = 4;
  }
  a.groups = (heads + a.heads_of_group - 1) / a.heads_of_group;
  a.threads = ((int64_t)T * a.groups) << a.lane_shift;
  return a;
}

template <typename Elem>
hipError_t launch(RotaryParams& p, hipStream_t stream) {
  const RotaryPlan a = rotary_plan(p.T, p.hq + p.hk + (p.cache.k ? p.hk : 0), p.d, p.rot);
  const unsigned blocks = (unsigned)ceil_div(a.threads, kThreads);
  p.groups = fast_div((uint32_t)a.groups);
  if (a.pieces) {
    p.units = p.d / 16;
    p.lane_shift = a.lane_shift;
    if (a.heads_of_group == 4) launch_units<Elem, 4>(p, blocks, stream);
    else launch_units<Elem, 1>(p, blocks, stream);
  } else {
    if (p.norm) hipLaunchKernelGGL((rotary_pairs_kernel<Elem, true>), dim3(blocks), dim3(kThreads), 0, stream, p);
    else hipLaunchKernelGGL((rotary_pairs_kernel<Elem, false>), dim3(blocks), dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

}  // namespace

bool rotary_fits(int32_t T, int heads, int32_t d, int32_t rot) {
  return rotary_plan(T, heads, d, rot).threads <= ((int64_t)1 << 32) - kThreads;
}

hipError_t launch_rotary(lora_dtype dt, RotaryParams p, hipStream_t stream) {
  switch (dt) {
    case LORA_F32: return launch<float>(p, stream);
    case LORA_F16: return launch<half_t>(p, stream);
    case LORA_BF16: return launch<bf16_t>(p, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_rope_table(const double* inv_freq, int32_t rot, double magnitude, int64_t first, int64_t n,
                             float* table, hipStream_t stream) {
  TableParams p{};
  p.table = table;
  p.first = first;
  p.n = n;
  p.magnitude = magnitude;
  p.half = rot / 2;
  p.by_half = fast_div((uint32_t)p.half);
  for (int i = 0; i < p.half; ++i) {
    p.turns[i] = inv_freq[i] / 6.283185307179586476925286766559;
    p.step[2 * i] = std::cos(inv_freq[i]);
    p.step[2 * i + 1] = std::sin(inv_freq[i]);
  }
  p.run = 8;
  while (ceil_div(n, p.run) * p.half > ((int64_t)1 << 30)) p.run *= 2;  // the kernel counts in 32 bits
  hipLaunchKernelGGL(rope_table_kernel, dim3((unsigned)ceil_div(ceil_div(n, p.run) * p.half, kThreads)), dim3(kThreads),
                     0, stream, p);
  return hipGetLastError();
}

}  // namespace lora
