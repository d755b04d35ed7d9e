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

__device__ inline bool names_page(int entry, int64_t n_pages) { return entry >= 0 && entry < n_pages; }

// ---- reserve ----------------------------------------------------------------

// The workspace of a reservation: [0, B) what each sequence lacks, then where its
// share of the free pages starts; [B] how many there are; from B + 1 on the pages.
__device__ inline int wanted_columns(const PoolParams& p, int tokens) {
  return tokens <= 0 ? 0 : min((int)p.page.div((uint32_t)(tokens - 1)) + 1, p.n_table);
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

// A workgroup: the row of fork i's child.
__device__ __forceinline__ void fork_row(const PoolParams& p, const ForkParams& f, int i) {
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
// used ones from it on, both ascending.  A wave looks at a range of a span of kSpan
// pages, 64 a load; lane i keeps the bits of the i-th load.  Workspace: the new
// number of each page from n_live on (-1: not in use).  8512 pages: 11.8 us (13.2
// with a scan of the workgroup for every 4096 pages).
constexpr int kOneWaves = kOne / 64;
constexpr int64_t kSpan = (int64_t)kOneWaves * 64 * 64;
__global__ __launch_bounds__(kOne) void compact_kernel(PoolParams p, int32_t* source, int32_t* target, int32_t* n_live,
                                                       int32_t* n_moves) {
  __shared__ int s_sums[2][kOneWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // of a span: the first page of this wave, and its loads
  struct Range {
    int64_t first;
    int loads;
  };
  const auto range_of = [&](int64_t span) {
    const int64_t pages = min(kSpan, p.n_pages - span);
    const int loads = (int)ceil_div(ceil_div(pages, 64), kOneWaves);
    return Range{span + (int64_t)wave * loads * 64, loads};
  };
  const auto used = [&](Range r) {
    uint64_t mine = 0;
    for (int i0 = 0; i0 < r.loads; i0 += 8) {
      int x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t page = r.first + 64 * (i0 + u) + lane;
        x[u] = i0 + u < r.loads && page < p.n_pages ? p.refs[page] : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const uint64_t bits = __ballot(x[u] > 0);
        if (lane == i0 + u) mine = bits;
      }
    }
    return mine;
  };
  // exclusive scan of two numbers over the workgroup's lanes
  const auto scan = [&](int (&x)[2], int (&total)[2]) {
    int up[2] = {x[0], x[1]};
#pragma unroll
    for (int o = 1; o < 64; o <<= 1)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int y = __shfl_up(up[k], o);
        if (lane >= o) up[k] += y;
      }
    __syncthreads();
    if (lane == 63) {
      s_sums[0][wave] = up[0];
      s_sums[1][wave] = up[1];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      x[k] = up[k] - x[k];
      total[k] = 0;
#pragma unroll
      for (int w = 0; w < kOneWaves; ++w) {
        if (w < wave) x[k] += s_sums[k][w];
        total[k] += s_sums[k][w];
      }
    }
  };
  int count[2] = {0, 0}, total[2];
  uint64_t bits = 0;
  for (int64_t span = 0; span < p.n_pages; span += kSpan) {
    bits = used(range_of(span));
    count[0] += __builtin_popcountll(bits);
  }
  scan(count, total);
  const int live = total[0];
  int at[2] = {0, 0};  // holes and moves so far
  for (int64_t span = 0; span < p.n_pages; span += kSpan) {
    const Range r = range_of(span);
    if (p.n_pages > kSpan) bits = used(r);
    // which of the lane's 64 pages are there, and which of them lie below n_live
    const auto below = [&](int64_t end) {
      const int64_t n = end - (r.first + 64 * lane);
      return lane >= r.loads || n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1);
    };
    const uint64_t there = below(p.n_pages), low = below(live);
    const uint64_t hole = ~bits & there & low, move = bits & ~low;
    int mine[2] = {__builtin_popcountll(hole), __builtin_popcountll(move)};
    scan(mine, total);
    for (int i = 0; i < r.loads; ++i) {
      const auto of_lane = [&](uint64_t x) {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, i) |
               ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), i) << 32);
      };
      const uint64_t holes = of_lane(hole), moves = of_lane(move);
      const int64_t page = r.first + 64 * i + lane;
      const auto rank = [&](uint64_t x) {
        return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(x >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)x, 0));
      };
      if (holes) {
        if ((holes >> lane) & 1) target[at[0] + __builtin_amdgcn_readlane(mine[0], i) + rank(holes)] = (int)page;
      }
      if (r.first + 64 * i + 63 >= live) {
        if ((moves >> lane) & 1) source[at[1] + __builtin_amdgcn_readlane(mine[1], i) + rank(moves)] = (int)page;
        else if (page >= live && page < p.n_pages) p.scratch[page] = -1;
      }
    }
    at[0] += total[0];
    at[1] += total[1];
  }
  __syncthreads();
  for (int i = (int)threadIdx.x; i < at[1]; i += kOne) {
    const int of = source[i], to = target[i];
    p.scratch[of] = to;
    p.refs[to] = p.refs[of];
    p.refs[of] = 0;
  }
  if (threadIdx.x == 0) {
    *n_live = live;
    *n_moves = at[1];
  }
}

// A workgroup: row b with the pages' new numbers.
__device__ __forceinline__ void rename_row(const PoolParams& p, int live, int b) {
  int32_t* row = p.table + b * p.ld_table;
  for (int c = threadIdx.x; c < p.n_table; c += kThreads) {
    const int entry = row[c];
    if (!names_page(entry, p.n_pages) || entry < live) continue;
    const int now = p.scratch[entry];
    if (now >= 0) row[c] = now;
  }
}

// ---- copy -------------------------------------------------------------------

// What a launch copies: the pages of up to kCopyTensors tensors, and beside them the
// rows that fork_row or rename_row writes (blockIdx.y past the tensors), which need
// what the copies need and nothing of them.
constexpr int kPiece = 1024;  // accesses of a workgroup at a time
template <typename Unit, bool STREAM>
__device__ __forceinline__ void copy_tensor(const MoveParams& p, const PagedTensor& t, int n) {
  const auto offset = [&](uint32_t u) {
    if (t.whole) return (int64_t)u * (int)sizeof(Unit);
    const uint32_t row = u / t.run, outer = row / t.n_inner;
    return (int64_t)outer * t.outer + (int64_t)(row - outer * t.n_inner) * t.inner + (int64_t)(u - row * t.run) * (int)sizeof(Unit);
  };
  const auto pages = [&](int pair, const char*& from, char*& to) {
    const int a = p.source[pair], b = p.target[pair];
    from = t.data + a * t.page;
    to = t.data + b * t.page;
    return names_page(a, p.n_pages) && names_page(b, p.n_pages);
  };
  constexpr int kEach = kPiece / kThreads;
  if (t.units >= (uint32_t)kPiece) {
    const int64_t pieces = ceil_div(t.units, kPiece);
    for (int64_t w = blockIdx.x; w < n * pieces; w += gridDim.x) {
      const int pair = (int)(w / pieces);
      const char* from;
      char* to;
      if (!pages(pair, from, to)) continue;
      const uint32_t u0 = (uint32_t)(w - pair * pieces) * kPiece + threadIdx.x;
      Unit x[kEach];
      int64_t at[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const uint32_t u = u0 + i * kThreads;
        at[i] = offset(u);
        if (u < t.units)
          x[i] = STREAM ? __builtin_nontemporal_load(reinterpret_cast<const Unit*>(from + at[i]))
                        : *reinterpret_cast<const Unit*>(from + at[i]);
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (u0 + i * kThreads < t.units) {
          Unit* dest = reinterpret_cast<Unit*>(to + at[i]);
          if constexpr (STREAM) __builtin_nontemporal_store(x[i], dest);
          else *dest = x[i];
        }
    }
  } else {
    // several small pages at a time
    const uint32_t at_once = kPiece / t.units;
    for (int64_t base = (int64_t)blockIdx.x * at_once; base < n; base += (int64_t)gridDim.x * at_once) {
      Unit x[kEach];
      char* dest[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const uint32_t q = threadIdx.x + i * kThreads, k = q / t.units;
        dest[i] = nullptr;
        if (k >= at_once || base + k >= n) continue;
        const char* from;
        char* to;
        if (!pages((int)(base + k), from, to)) continue;
        const int64_t at = offset(q - k * t.units);
        x[i] = *reinterpret_cast<const Unit*>(from + at);
        dest[i] = to + at;
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (dest[i]) *reinterpret_cast<Unit*>(dest[i]) = x[i];
    }
  }
}

template <bool STREAM>
__global__ __launch_bounds__(kThreads) void move_kernel(MoveParams p) {
  if ((int)blockIdx.y == p.n_tensors) {
    if (p.task == MoveParams::kFork) {
      for (int i = blockIdx.x; i < p.fork.n; i += gridDim.x) fork_row(p.pool, p.fork, i);
    } else {
      const int live = *p.n_live;
      for (int b = blockIdx.x; b < p.pool.B; b += gridDim.x) rename_row(p.pool, live, b);
    }
    return;
  }
  int n = p.n;
  if (p.count) n = min(n, *p.count);
  const PagedTensor& t = p.t[blockIdx.y];
  if (t.unit == 16) copy_tensor<u32x4, STREAM>(p, t, n);
  else if (t.unit == 4) copy_tensor<uint32_t, STREAM>(p, t, n);
  else copy_tensor<uint8_t, STREAM>(p, t, n);
}

dim3 rows4(int64_t rows) { return dim3((unsigned)ceil_div(rows, kThreads / 64)); }

}  // namespace

int64_t pages_scratch_bytes(int64_t n_pages, int32_t n_seqs) { return 4 * (n_pages + (int64_t)n_seqs + 1); }

hipError_t launch_reserve(const PoolParams& p, const int32_t* lengths, int32_t* missing, hipStream_t stream) {
  if (p.B > 0) hipLaunchKernelGGL(count_missing_kernel, rows4(p.B), dim3(kThreads), 0, stream, p, lengths);
  hipLaunchKernelGGL(take_pages_kernel, dim3(1), dim3(kOne), 0, stream, p, missing);
  if (p.B > 0) hipLaunchKernelGGL(hand_out_kernel, rows4(p.B), dim3(kThreads), 0, stream, p, lengths);
  return hipGetLastError();
}

hipError_t launch_fork(const PoolParams& p, const ForkParams& f, hipStream_t stream) {
  hipLaunchKernelGGL(fork_pages_kernel, dim3(1), dim3(kOne), 0, stream, p, f);
  return hipGetLastError();
}

hipError_t launch_release(const PoolParams& p, const int32_t* rows, const int32_t* keep, int32_t n, hipStream_t stream) {
  hipLaunchKernelGGL(release_kernel, dim3((unsigned)n), dim3(kThreads), 0, stream, p, rows, keep);
  return hipGetLastError();
}

hipError_t launch_compact(const PoolParams& p, int32_t* source, int32_t* target, int32_t* n_live, int32_t* n_moves,
                          hipStream_t stream) {
  hipLaunchKernelGGL(compact_kernel, dim3(1), dim3(kOne), 0, stream, p, source, target, n_live, n_moves);
  return hipGetLastError();
}

hipError_t launch_move(const MoveParams& p, hipStream_t stream) {
  int64_t most = p.task == MoveParams::kFork ? p.fork.n : p.task == MoveParams::kRename ? p.pool.B : 0;
  int64_t bytes = 0;  // read and written at most
  for (int i = 0; i < p.n_tensors; ++i) {
    const uint32_t units = p.t[i].units;
    bytes += 2 * (int64_t)units * p.t[i].unit * p.n;
    most = std::max(most, units >= (uint32_t)kPiece ? ceil_div(units, kPiece) * p.n : ceil_div(p.n, kPiece / units));
  }
  const int rows = p.n_tensors + (p.task ? 1 : 0);
  if (rows == 0 || most == 0) return hipSuccess;
  // some 16 workgroups a compute unit in all
  const dim3 grid((unsigned)std::min<int64_t>(most, std::max(4096 / rows, 64)), (unsigned)rows);
  // More than the last-level cache (256 MB) holds goes past the caches: 187 us for 196 to
  // 205 for 0.83 GB, where 0.13 GB took 41 us for 38.  The host knows the most that may
  // move, half of a pool, not what does.
  if (bytes > (int64_t)1 << 29) hipLaunchKernelGGL(move_kernel<true>, grid, dim3(kThreads), 0, stream, p);
  else hipLaunchKernelGGL(move_kernel<false>, grid, dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace lora
