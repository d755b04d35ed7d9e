// What a tree of drafted tokens needs around its attention: the ancestor
// masks, positions and cache rows of a step (once for all layers), and the
// move of the accepted path's cache rows to the end of the context.
#include "attention.h"

namespace lora {

namespace {

constexpr int kThreads = 256;

// One workgroup a sequence.  A node's mask row is its own bit and those of the
// nodes on its way to the context; the parents are staged in LDS, and each
// thread walks its node's way once, up to the node's depth.  A parent is
// smaller than its node, so every walk ends.
__global__ __launch_bounds__(kThreads) void build_tree_kernel(BuildTreeParams p) {
  warm_args(p);
  __shared__ int s_parent[LORA_MAX_TREE_NODES];
  const int b = blockIdx.x;
  const int64_t start = p.q_start[b];
  int64_t n = (int64_t)p.q_start[b + 1] - start;
  if (start < 0 || start > p.T) return;
  n = n < 0 ? 0 : (n > p.max_nodes ? p.max_nodes : n);
  if (n > p.T - start) n = p.T - start;
  const int64_t ctx = p.context[b] < 0 ? 0 : p.context[b];
  if (p.parents) {
    for (int j = threadIdx.x; j < n; j += kThreads) {
      const int q = p.parents[start + j];
      s_parent[j] = q >= 0 && q < j ? q : -1;
    }
    __syncthreads();
  }
  for (int64_t j = threadIdx.x; j < n; j += kThreads) {
    const int64_t row = start + j;
    int64_t depth = j;
    uint64_t* bits = p.mask ? p.mask + row * p.mask_words : nullptr;
    if (!p.parents) {
      if (bits)
        for (int w = 0; w < p.mask_words; ++w)
          bits[w] = j >= 64 * (int64_t)w + 63 ? ~0ull : (j < 64 * (int64_t)w ? 0ull : ~0ull >> (63 - (j & 63)));
    } else {
      depth = 0;
      // the way visits descending nodes: each word is complete when the way
      // leaves it
      int at = (int)j;
      int word = p.mask_words;
      uint64_t cur = 0;
      if (bits)
        for (int w = (at >> 6) + 1; w < p.mask_words; ++w) bits[w] = 0;
      word = at >> 6;
      while (true) {
        if ((at >> 6) != word) {
          if (bits) {
            bits[word] = cur;
            for (int w = (at >> 6) + 1; w < word; ++w) bits[w] = 0;
          }
          word = at >> 6;
          cur = 0;
        }
        cur |= 1ull << (at & 63);
        at = s_parent[at];
        if (at < 0) break;
        ++depth;
      }
      if (bits) {
        bits[word] = cur;
        for (int w = 0; w < word; ++w) bits[w] = 0;
      }
    }
    if (p.positions) p.positions[row] = (int)(ctx + depth);
    if (p.cache_rows) {
      const int64_t pos = ctx + j;
      int got = -1;
      if (pos < (int64_t)1 << 31) {
        const int64_t col = p.page.div((uint32_t)pos);
        if (col < p.n_table) {
          const int64_t page = p.page_table[b * p.ld_table + col];
          if (page >= 0 && page < p.n_pages) got = (int)(page * p.page.d + (pos - col * p.page.d));
        }
      }
      p.cache_rows[row] = got;
    }
  }
}

// One workgroup a (layer's K or V, kKeepHeads heads, sequence).  Destination j never lies
// past its source path[j] >= j, and the sources ascend, so taking the entries
// in rounds, each read whole before it is written, never overwrites a row that
// is still to be read.  All layers are one launch.  A head's rows are some 1 KB, far
// less than a workgroup costs to start: 64 sequences, 16 layers of 8 bf16 heads of
// 128 (34 MB) took 23.8 us with a workgroup each, 16.0 with four heads in one.
constexpr int kKeepHeads = 4;
__global__ __launch_bounds__(kThreads) void keep_path_kernel(KeepParams p, int kv_heads) {
  const int b = blockIdx.x, h0 = (int)blockIdx.y * kKeepHeads, z = blockIdx.z;
  const int layer = z >> 1;
  const int64_t head_b = z & 1 ? p.v_head : p.k_head;
  char* base = static_cast<char*>(z & 1 ? p.v[layer] : p.k[layer]) + h0 * head_b;
  const int64_t page_b = z & 1 ? p.v_page : p.k_page, row_b = z & 1 ? p.v_row : p.k_row;
  const int64_t ctx = p.context[b];
  int n = p.n_kept[b];
  n = n > p.n_path ? p.n_path : n;
  if (ctx < 0 || n <= 0) return;
  const int32_t* path = p.path + b * p.ld_path;
  // the path ends before the first entry that does not ascend
  const int lane = threadIdx.x & 63;
  for (int j0 = 0; j0 < n; j0 += 64) {
    const int j = j0 + lane;
    const bool bad = j < n && path[j] <= (j ? path[j - 1] : -1);
    const unsigned long long any = __ballot(bad);
    if (any) {
      n = j0 + __builtin_ctzll(any);
      break;
    }
  }
  const int pieces = p.row_bytes / 16, rows = kThreads / pieces;
  const int r = threadIdx.x / pieces, c = threadIdx.x - r * pieces;
  auto at = [&](int64_t pos) -> char* {
    if (pos >= (int64_t)1 << 31) return nullptr;
    const int64_t col = p.page.div((uint32_t)pos);
    if (col >= p.n_table) return nullptr;
    const int64_t page = p.page_table[b * p.ld_table + col];
    if (page < 0 || page >= p.n_pages) return nullptr;
    return base + page * page_b + (pos - col * p.page.d) * row_b + 16 * c;
  };
  for (int j0 = 0; j0 < n; j0 += rows) {
    const int j = j0 + r;
    u32x4 x[kKeepHeads];
    const char* of = nullptr;
    char* to = nullptr;
    if (r < rows && j < n && path[j] != j) {
      of = at(ctx + path[j]);
      to = of ? at(ctx + j) : nullptr;
    }
    if (to)
#pragma unroll
      for (int i = 0; i < kKeepHeads; ++i)  // (past the last head: the last again)
        x[i] = *reinterpret_cast<const u32x4*>(of + min(i, kv_heads - 1 - h0) * head_b);
    __syncthreads();
    if (to)
#pragma unroll
      for (int i = 0; i < kKeepHeads; ++i)
        if (h0 + i < kv_heads) *reinterpret_cast<u32x4*>(to + i * head_b) = x[i];
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_build_tree(const BuildTreeParams& p, hipStream_t stream) {
  hipLaunchKernelGGL(build_tree_kernel, dim3((unsigned)p.B), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

hipError_t launch_keep_path(const KeepParams& p, int32_t n_layers, int32_t kv_heads, int32_t B, hipStream_t stream) {
  hipLaunchKernelGGL(keep_path_kernel, 
                     dim3((unsigned)B, (unsigned)ceil_div(kv_heads, kKeepHeads), (unsigned)(2 * n_layers)),
                     dim3(kThreads), 0, stream, p, kv_heads);
  return hipGetLastError();
}

}  // namespace lora
