// Attention of a step's drafted tokens over the paged cache.
//
// One wave a (token, query head): the lanes hold the query, take the keys one
// after another and keep the running maximum and sum of the softmax.
#include "attention.h"

namespace lora {

namespace {

template <typename Elem>
__global__ __launch_bounds__(64) void attend_kernel(AttendParams p) {
  warm_args(p);
  const int b = blockIdx.z, h = blockIdx.y, i = blockIdx.x, lane = threadIdx.x;
  const int start = p.q_start[b];
  int n = p.q_start[b + 1] - start;
  if (start < 0 || start > p.T) return;
  n = n > p.max_nodes ? p.max_nodes : n;
  n = n > p.T - start ? p.T - start : n;
  if (i >= n) return;
  int ctx = p.context[b];
  ctx = ctx < 0 ? 0 : (ctx > p.max_context ? p.max_context : ctx);
  const int64_t row = start + i;
  const int kv = p.group.div(h);
  const Elem* q = static_cast<const Elem*>(p.q) + row * p.ldq + (int64_t)h * p.d;
  float qf[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) qf[e] = lane + 64 * e < p.d ? (float)q[lane + 64 * e] : 0.f;
  for (int64_t pos = 0; pos < (int64_t)ctx + n; ++pos) {
    const int64_t j = pos - ctx;
    if (j >= 0) {
      if (!p.mask) {
        if (j > i) break;
      } else if (!(p.mask[row * p.mask_words + (j >> 6)] >> (j & 63) & 1)) {
        continue;
      }
    }
    const int64_t col = p.cache.page.div((uint32_t)pos);
    if (col >= p.n_table) break;
    const int64_t page = p.page_table[b * p.ld_table + col];
    if (page < 0 || page >= p.cache.n_pages) continue;
    const int64_t place = pos - col * p.cache.page.d;
    const Elem* k = static_cast<const Elem*>(p.cache.k) + page * p.cache.k_page + kv * p.cache.k_head + place * p.cache.k_row;
    const Elem* v = static_cast<const Elem*>(p.cache.v) + page * p.cache.v_page + kv * p.cache.v_head + place * p.cache.v_row;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 64 * e < p.d) s = __builtin_fmaf(qf[e], (float)k[lane + 64 * e], s);
#pragma unroll
    for (int w = 32; w; w >>= 1) s += __shfl_xor(s, w);
    s *= p.scale;
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), f = __expf(m - mn), wgt = __expf(s - mn);
    m = mn;
    l = l * f + wgt;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + 64 * e < p.d) o[e] = o[e] * f + wgt * (float)v[lane + 64 * e];
  }
  Elem* out = static_cast<Elem*>(p.out) + row * p.ldo + (int64_t)h * p.d;
  const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + 64 * e < p.d) out[lane + 64 * e] = static_cast<Elem>(o[e] * inv);
  if (p.lse && lane == 0) p.lse[row * p.hq + h] = m + logf(l);
}

template <typename Elem>
hipError_t launch(const AttendParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(attend_kernel<Elem>, dim3((unsigned)p.max_nodes, (unsigned)p.hq, (unsigned)p.B), dim3(64), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace

int64_t attend_need_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

hipError_t launch_attend(lora_dtype dt, const AttendParams& p, hipStream_t stream) {
  switch (dt) {
    case LORA_F32: return launch<float>(p, stream);
    case LORA_F16: return launch<half_t>(p, stream);
    case LORA_BF16: return launch<bf16_t>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace lora
