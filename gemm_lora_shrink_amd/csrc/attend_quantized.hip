// Attention of a step's tokens over a quantized cache: a wave a row and query
// head, one key a lane for the scores, four elements a lane for the values.
#include "cache.h"

namespace lora {

namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

template <typename Elem, typename F>
__global__ __launch_bounds__(kThreads) void attend_quantized_kernel(AttendQuantizedParams p) {
  warm_args(p);
  __shared__ float s_q[kWaves][256];
  __shared__ float s_w[kWaves][64];
  __shared__ const char* s_row[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int b = blockIdx.y, r = (int)blockIdx.x * kWaves + wave;
  const int i = r / p.hq, h = r - i * p.hq;
  const int64_t start = p.q_start[b];
  int64_t n = (int64_t)p.q_start[b + 1] - start;
  if (start < 0 || start > p.T) return;
  n = n > p.T - start ? p.T - start : n;
  n = n > p.max_nodes ? p.max_nodes : n;
  if (i >= n) return;
  int64_t ctx = p.context[b];
  ctx = ctx < 0 ? 0 : (ctx > p.max_context ? p.max_context : ctx);
  const int64_t row = start + i;
  const int kv = (int)p.group.div((uint32_t)h);
  const QuantizedView& c = p.cache;
  const Elem* q = static_cast<const Elem*>(p.q) + row * p.ldq + (int64_t)h * p.d;
  for (int e = lane; e < p.d; e += 64) {
    uint32_t bits;
    if constexpr (sizeof(Elem) == 4) bits = reinterpret_cast<const uint32_t*>(q)[e];
    else bits = reinterpret_cast<const uint16_t*>(q)[e];
    s_q[wave][e] = Traits<Elem>::elem_to_float(bits) * p.scale * kLog2e;
  }
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int64_t end = ctx + (p.mask ? n : i + 1);
  const int at = 4 * lane;
  for (int64_t k0 = 0; k0 < end; k0 += 64) {
    const int64_t pos = k0 + lane;
    float s = -INFINITY, v_scale = 0.f;
    const char* v_row = nullptr;
    bool seen = pos < end;
    if (seen && pos >= ctx && p.mask) {
      const int64_t node = pos - ctx;
      seen = (node >> 6) < p.mask_words && (p.mask[row * p.mask_words + (node >> 6)] >> (node & 63) & 1);
    }
    if (seen) {
      const int64_t col = c.page.div((uint32_t)pos);
      const int64_t page = col < p.n_table ? p.page_table[b * p.ld_table + col] : -1;
      seen = page >= 0 && page < c.n_pages;
      if (seen) {
        const int place = (int)(pos - col * c.page.d), block = (int)c.block.div((uint32_t)place);
        const char* k_row = static_cast<const char*>(c.k) + page * c.k_page + kv * c.k_head + place * c.k_row;
        v_row = static_cast<const char*>(c.v) + page * c.v_page + kv * c.v_head + place * c.v_row;
        v_scale = power_of_two(exponent_of<F>(c.v_exp[page * c.v_exp_page + kv * c.v_exp_head + block]));
        float sum = 0.f;
        for (int e = 0; e < p.d; e += 4) {
          float x[4];
          F::numbers(*reinterpret_cast<const uint32_t*>(k_row + e), x);
          for (int j = 0; j < 4; ++j) sum = __builtin_fmaf(x[j], s_q[wave][e + j], sum);
        }
        s = sum * power_of_two(exponent_of<F>(c.k_exp[page * c.k_exp_page + kv * c.k_exp_head + block]));
      }
    }
    float mx = s;
    for (int x = 32; x; x >>= 1) mx = fmaxf(mx, __shfl_xor(mx, x));
    const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.f : mn;
    const float f = __builtin_amdgcn_exp2f(m - ms);
    const float w = seen ? __builtin_amdgcn_exp2f(s - ms) : 0.f;
    m = mn;
    float sum = w;
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * f + sum;
    for (int e = 0; e < 4; ++e) o[e] *= f;
    s_w[wave][lane] = w * v_scale;
    s_row[wave][lane] = v_row;
    __builtin_amdgcn_wave_barrier();
    if (at < p.d)
      for (int j = 0; j < 64; ++j) {
        const char* vr = s_row[wave][j];
        if (!vr) continue;
        float x[4];
        F::numbers(*reinterpret_cast<const uint32_t*>(vr + at), x);
        for (int e = 0; e < 4; ++e) o[e] = __builtin_fmaf(s_w[wave][j], x[e], o[e]);
      }
    __builtin_amdgcn_wave_barrier();
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  Elem* out = static_cast<Elem*>(p.out) + row * p.ldo + (int64_t)h * p.d;
  if (at < p.d)
    for (int e = 0; e < 4; ++e) out[at + e] = static_cast<Elem>(o[e] * inv);
  if (p.lse && lane == 0) p.lse[row * p.hq + h] = (m + __builtin_amdgcn_logf(l)) * kLn2;
}

int64_t grid_of(int32_t max_nodes, int32_t hq) { return ceil_div((int64_t)max_nodes * hq, kWaves); }

template <typename Elem>
hipError_t launch(int format, const AttendQuantizedParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)grid_of(p.max_nodes, p.hq), (unsigned)p.B);
  if (format == LORA_CACHE_E4M3)
    hipLaunchKernelGGL((attend_quantized_kernel<Elem, E4m3>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((attend_quantized_kernel<Elem, Int8>), grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace

bool attend_quantized_fits(lora_dtype, int32_t, int32_t max_nodes, int32_t, int32_t hq, int32_t, int32_t) {
  return grid_of(max_nodes, hq) <= (((int64_t)1 << 32) - 1) / kThreads;
}
int64_t attend_quantized_need_bytes(lora_dtype, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) {
  return 0;
}
int64_t attend_quantized_most_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_attend_quantized(lora_dtype dt, int format, const AttendQuantizedParams& p, hipStream_t stream) {
  switch (dt) {
    case LORA_F32: return launch<float>(format, p, stream);
    case LORA_F16: return launch<half_t>(format, p, stream);
    case LORA_BF16: return launch<bf16_t>(format, p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace lora
