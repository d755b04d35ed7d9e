// The pages of a cache: who holds them (reserve, fork, release, compact), and
// copying them.
//
// Reference counts and tables are small (a pool of 100 000 pages is 400 KB), so
// what has an order (which free page goes to whom) is done by one workgroup with
// scans, and what has none by as many as there are rows.  The calls are a few
// microseconds; the copies move the bytes.
#include <algorithm>

#include "cache.h"

namespace lora {

namespace {

constexpr int kOne = 1024;      // threads of the workgroup that keeps the order
constexpr int kThreads = 256;   // of the others

// Exclusive scan over the workgroup of each thread's flag bits: thread t's
// predecessors' number of ones; total: all of them.  Four flags a thread.
struct Scan {
  int* wave_sums;  // [kOne / 64] in LDS
  __device__ __forceinline__ int flags(uint32_t four, int& total) {
    int before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t b = __ballot((four >> k) & 1);
      before += __builtin_amdgcn_mbcnt_hi((uint32_t)(b >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)b, 0));
      all += __builtin_popcountll(b);
    }
    return spread(before, all, total);
  }
  __device__ __forceinline__ int numbers(int x, int& total) {
    int up = x;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(up, o);
      if ((int)(threadIdx.x & 63) >= o) up += y;
    }
    return spread(up - x, __shfl(up, 63), total);
  }
  __device__ __forceinline__ int spread(int before, int all, int& total) {
    const int wave = threadIdx.x >> 6;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) wave_sums[wave] = all;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kOne / 64; ++w) {
      if (w < wave) before += wave_sums[w];
      sum += wave_sums[w];
    }
    total = sum;
    return before;
  }
};

// The first `want` free pages in ascending order go to take(rank, page); returns how
// many there were.  Called by the whole workgroup.
template <typename Take>
__device__ __forceinline__ int free_pages(Scan& scan, const int32_t* refs, int64_t n_pages, int want, Take take) {
  int found = 0;
  for (int64_t p0 = 0; p0 < n_pages && found < want; p0 += 4 * kOne) {
    const int64_t mine = p0 + 4 * (int)threadIdx.x;
    uint32_t four = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (mine + k < n_pages && refs[mine + k] <= 0) four |= 1u << k;
    int total;
    int rank = found + scan.flags(four, total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((four >> k) & 1) {
        if (rank < want) take(rank, (int)(mine + k));
        ++rank;
      }
    found += total;
  }
  return min(found, want);
}

__device__ inline int clamped(int64_t x, int64_t hi) { return (int)(x < 0 ? 0 : (x > hi ? hi : x)); }
__device__ inline bool names_page(int entry, int64_t n_pages) { return entry >= 0 && entry < n_pages; }

// ---- reserve ----------------------------------------------------------------

// The workspace of a reservation: [0, B) what each sequence lacks, then where its
// share of the free pages starts; [B] how many there are; from B + 1 on the pages.
__device__ inline int wanted_columns(const PoolParams& p, int64_t tokens) {
  return clamped((int64_t)p.page.div((uint32_t)clamped(tokens + p.page.d - 1, 0x7fffffff)), p.n_table);
}

__global__ __launch_bounds__(kThreads) void count_missing_kernel(PoolParams p, const int32_t* lengths) {
  const int b = (int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (b >= p.B) return;
  const int cols = wanted_columns(p, lengths[b]);
  int n = 0;
  for (int c0 = 0; c0 < cols; c0 += 64) {
    const bool lacks = c0 + lane < cols && !names_page(p.table[b * p.ld_table + c0 + lane], p.n_pages);
    n += __builtin_popcountll(__ballot(lacks));
  }
  if (lane == 0) p.scratch[b] = n;
}

__global__ __launch_bounds__(kOne) void take_pages_kernel(PoolParams p, int32_t* missing) {
  __shared__ int sums[kOne / 64];
  Scan scan{sums};
  int want = 0;
  for (int b0 = 0; b0 < p.B; b0 += kOne) {
    const int b = b0 + (int)threadIdx.x;
    const int n = b < p.B ? p.scratch[b] : 0;
    int total;
    const int before = scan.numbers(n, total);
    if (b < p.B) p.scratch[b] = want + before;
    want += total;
  }
  int32_t* pages = p.scratch + p.B + 1;
  const int got = free_pages(scan, p.refs, p.n_pages, want, [&](int rank, int page) {
    pages[rank] = page;
    p.refs[page] = 1;
  });
  if (threadIdx.x == 0) {
    p.scratch[p.B] = got;
    if (missing) *missing = want - got;
  }
}

__global__ __launch_bounds__(kThreads) void hand_out_kernel(PoolParams p, const int32_t* lengths) {
  const int b = (int)blockIdx.x * (kThreads / 64) + (int)(threadIdx.x >> 6), lane = threadIdx.x & 63;
  if (b >= p.B) return;
  const int cols = wanted_columns(p, lengths[b]), got = p.scratch[p.B];
  int at = p.scratch[b];
  const int32_t* pages = p.scratch + p.B + 1;
  for (int c0 = 0; c0 < cols; c0 += 64) {
    int32_t* entry = p.table + b * p.ld_table + c0 + lane;
    const bool lacks = c0 + lane < cols && !names_page(*entry, p.n_pages);
    const uint64_t all = __ballot(lacks);
    const int rank = at + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
    if (lacks) *entry = rank < got ? pages[rank] : -1;
    at += __builtin_popcountll(all);
  }
}

// ---- fork -------------------------------------------------------------------

// One workgroup: which forks need a page for the tokens that fill one in part, and
// which page each gets.  Workspace: the rank of each fork's page (-1: none needed),
// then the pages.
__global__ __launch_bounds__(kOne) void fork_pages_kernel(PoolParams p, ForkParams f) {
  __shared__ int sums[kOne / 64];
  Scan scan{sums};
  int want = 0;
  for (int i0 = 0; i0 < f.n; i0 += kOne) {
    const int i = i0 + (int)threadIdx.x;
    int of = -1;
    if (i < f.n) {
      const int parent = f.parents[i], child = f.children[i], n = f.lengths[i];
      if (parent >= 0 && parent < f.B_from && child >= 0 && child < p.B && n > 0) {
        const int full = (int)p.page.div((uint32_t)n);
        if (full < p.n_table && n - full * (int)p.page.d > 0) of = f.from[parent * f.ld_from + full];
        if (!names_page(of, p.n_pages)) of = -1;
      }
    }
    int total;
    const int rank = want + scan.flags(of >= 0 ? 1u : 0u, total);
    if (i < f.n) {
      f.source[i] = of;
      p.scratch[i] = of >= 0 ? rank : -1;
    }
    want += total;
  }
  int32_t* pages = p.scratch + f.n;
  const int got = free_pages(scan, p.refs, p.n_pages, want, [&](int rank, int page) {
    pages[rank] = page;
    p.refs[page] = 1;
  });
  __syncthreads();
  for (int i = (int)threadIdx.x; i < f.n; i += kOne) {
    const int rank = p.scratch[i];
    const bool has = rank >= 0 && rank < got;
    f.target[i] = has ? pages[rank] : -1;
    if (!has) f.source[i] = -1;
  }
  if (f.missing && threadIdx.x == 0) *f.missing = want - got;
}

// A workgroup a fork: the child's row.
__global__ __launch_bounds__(kThreads) void fork_rows_kernel(PoolParams p, ForkParams f) {
  const int i = blockIdx.x;
  const int parent = f.parents[i], child = f.children[i];
  if (child < 0 || child >= p.B) return;
  const int n = parent >= 0 && parent < f.B_from ? max(f.lengths[i], 0) : 0;
  const int full = (int)p.page.div((uint32_t)n), target = f.target[i];
  const int32_t* from = f.from + (n ? parent : 0) * f.ld_from;
  int32_t* to = p.table + child * p.ld_table;
  for (int c = threadIdx.x; c < p.n_table; c += kThreads) {
    int entry = -1;
    if (c < full) {
      entry = from[c];
      if (names_page(entry, p.n_pages)) atomicAdd(p.refs + entry, 1);
      else entry = -1;
    } else if (c == full) {
      entry = target;
    }
    to[c] = entry;
  }
}

// ---- release ----------------------------------------------------------------

// A workgroup a row.  Entries are exchanged for -1, so a row that is listed twice
// gives each page back once.
__global__ __launch_bounds__(kThreads) void release_kernel(PoolParams p, const int32_t* rows, const int32_t* keep) {
  const int i = blockIdx.x;
  const int b = rows ? rows[i] : i;
  if (b < 0 || b >= p.B) return;
  const int first = keep ? wanted_columns(p, keep[i]) : 0;
  for (int c = first + (int)threadIdx.x; c < p.n_table; c += kThreads) {
    const int entry = atomicExch(p.table + b * p.ld_table + c, -1);
    if (names_page(entry, p.n_pages)) atomicSub(p.refs + entry, 1);
  }
}

// ---- compact ----------------------------------------------------------------

// One workgroup: the number of pages in use, then the free ones below it and the
// used ones from it on, both ascending.  Workspace: the new number of each page
// from n_live on (-1: not in use).
__global__ __launch_bounds__(kOne) void compact_kernel(PoolParams p, int32_t* source, int32_t* target, int32_t* n_live,
                                                       int32_t* n_moves) {
  __shared__ int sums[kOne / 64];
  Scan scan{sums};
  int live = 0;
  for (int64_t p0 = 0; p0 < p.n_pages; p0 += 4 * kOne) {
    const int64_t mine = p0 + 4 * (int)threadIdx.x;
    uint32_t four = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (mine + k < p.n_pages && p.refs[mine + k] > 0) four |= 1u << k;
    int total;
    scan.flags(four, total);
    live += total;
  }
  int holes = 0, moves = 0;
  for (int64_t p0 = 0; p0 < p.n_pages; p0 += 4 * kOne) {
    const int64_t mine = p0 + 4 * (int)threadIdx.x;
    uint32_t hole = 0, move = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t page = mine + k;
      if (page >= p.n_pages) continue;
      const bool used = p.refs[page] > 0;
      if (!used && page < live) hole |= 1u << k;
      if (used && page >= live) move |= 1u << k;
      if (page >= live) p.scratch[page] = -1;
    }
    int total;
    int at = holes + scan.flags(hole, total);
    holes += total;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((hole >> k) & 1) target[at++] = (int)(mine + k);
    at = moves + scan.flags(move, total);
    moves += total;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((move >> k) & 1) source[at++] = (int)(mine + k);
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < moves; i += kOne) {
    const int of = source[i], to = target[i];
    p.scratch[of] = to;
    p.refs[to] = p.refs[of];
    p.refs[of] = 0;
  }
  if (threadIdx.x == 0) {
    *n_live = live;
    *n_moves = moves;
  }
}

__global__ __launch_bounds__(kThreads) void rename_kernel(PoolParams p, const int32_t* n_live) {
  const int live = *n_live;
  int32_t* row = p.table + (int64_t)blockIdx.x * p.ld_table;
  for (int c = threadIdx.x; c < p.n_table; c += kThreads) {
    const int entry = row[c];
    if (!names_page(entry, p.n_pages) || entry < live) continue;
    const int now = p.scratch[entry];
    if (now >= 0) row[c] = now;
  }
}

// ---- copy -------------------------------------------------------------------

// A workgroup takes pieces of 1024 accesses of one tensor, pair after pair.
constexpr int kPiece = 1024;
template <typename Unit>
__global__ __launch_bounds__(kThreads) void copy_pages_kernel(CopyParams p) {
  const lora_paged_tensor& t = p.t[blockIdx.y];
  int n = p.n;
  if (p.count) n = min(n, *p.count);
  const int64_t run = t.run / (int)sizeof(Unit), units = run * t.n_inner * t.n_outer;
  const int64_t pieces = ceil_div(units, kPiece);
  const bool whole = t.n_inner == 1 && t.n_outer == 1;
  for (int64_t w = blockIdx.x; w < n * pieces; w += gridDim.x) {
    const int pair = (int)(w / pieces);
    const int of = p.source[pair], to = p.target[pair];
    if (!names_page(of, p.n_pages) || !names_page(to, p.n_pages)) continue;
    const char* from = static_cast<const char*>(t.data) + of * t.page;
    char* dest = static_cast<char*>(t.data) + to * t.page;
    const int64_t u0 = (w - pair * pieces) * kPiece + threadIdx.x;
    Unit x[kPiece / kThreads];
    int64_t at[kPiece / kThreads];
#pragma unroll
    for (int i = 0; i < kPiece / kThreads; ++i) {
      const int64_t u = u0 + i * kThreads;
      if (whole) {
        at[i] = u * (int64_t)sizeof(Unit);
      } else {
        const int64_t row = u / run, outer = row / t.n_inner;
        at[i] = outer * t.outer + (row - outer * t.n_inner) * t.inner + (u - row * run) * (int64_t)sizeof(Unit);
      }
      if (u < units) x[i] = *reinterpret_cast<const Unit*>(from + at[i]);
    }
#pragma unroll
    for (int i = 0; i < kPiece / kThreads; ++i)
      if (u0 + i * kThreads < units) *reinterpret_cast<Unit*>(dest + at[i]) = x[i];
  }
}

dim3 rows4(int64_t rows) { return dim3((unsigned)ceil_div(rows, kThreads / 64)); }

}  // namespace

int64_t pages_scratch_bytes(int64_t n_pages, int32_t n_seqs) { return 4 * (n_pages + (int64_t)n_seqs + 1); }

hipError_t launch_reserve(const PoolParams& p, const int32_t* lengths, int32_t* missing, hipStream_t stream) {
  hipLaunchKernelGGL(count_missing_kernel, rows4(p.B), dim3(kThreads), 0, stream, p, lengths);
  hipLaunchKernelGGL(take_pages_kernel, dim3(1), dim3(kOne), 0, stream, p, missing);
  hipLaunchKernelGGL(hand_out_kernel, rows4(p.B), dim3(kThreads), 0, stream, p, lengths);
  return hipGetLastError();
}

hipError_t launch_fork(const PoolParams& p, const ForkParams& f, hipStream_t stream) {
  hipLaunchKernelGGL(fork_pages_kernel, dim3(1), dim3(kOne), 0, stream, p, f);
  hipLaunchKernelGGL(fork_rows_kernel, dim3((unsigned)f.n), dim3(kThreads), 0, stream, p, f);
  return hipGetLastError();
}

hipError_t launch_release(const PoolParams& p, const int32_t* rows, const int32_t* keep, int32_t n, hipStream_t stream) {
  hipLaunchKernelGGL(release_kernel, dim3((unsigned)n), dim3(kThreads), 0, stream, p, rows, keep);
  return hipGetLastError();
}

hipError_t launch_compact(const PoolParams& p, int32_t* source, int32_t* target, int32_t* n_live, int32_t* n_moves,
                          hipStream_t stream) {
  hipLaunchKernelGGL(compact_kernel, dim3(1), dim3(kOne), 0, stream, p, source, target, n_live, n_moves);
  if (p.B > 0) hipLaunchKernelGGL(rename_kernel, dim3((unsigned)p.B), dim3(kThreads), 0, stream, p, n_live);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const CopyParams& p, int32_t n_tensors, hipStream_t stream) {
  // some 16 workgroups a compute unit in all
  int64_t most = 0;
  for (int i = 0; i < n_tensors; ++i) {
    const lora_paged_tensor& t = p.t[i];
    most = std::max(most, ceil_div((int64_t)(t.run / p.unit) * t.n_inner * t.n_outer, kPiece) * p.n);
  }
  const dim3 grid((unsigned)std::min<int64_t>(most, std::max(4096 / n_tensors, 64)), (unsigned)n_tensors);
  if (p.unit == 16) hipLaunchKernelGGL(copy_pages_kernel<u32x4>, grid, dim3(kThreads), 0, stream, p);
  else if (p.unit == 4) hipLaunchKernelGGL(copy_pages_kernel<uint32_t>, grid, dim3(kThreads), 0, stream, p);
  else hipLaunchKernelGGL(copy_pages_kernel<uint8_t>, grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace lora
