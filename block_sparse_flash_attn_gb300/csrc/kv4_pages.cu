// Pages of the 4-bit cache: copied, given to sequences that grow, shared by
// sequences that fork, and moved together.
//
// refs[p] is the number of block-table rows that hold page p; a page that none
// holds is free.  A page that is not full belongs to one row, so that tokens
// are written to no other row's page.  What is given out is the lowest free page,
// in the order of rows and columns: the results are a function of the arguments,
// whatever order threads run in.
//
// Bound: launches and dependent loads for the books (refs and tables are some
// hundred KB at most), memory for the pages that move.
#include <algorithm>
#include <cstdint>

#include "kv4.cuh"

namespace bsattn {
namespace {

constexpr int kRowsThreads = 128;
constexpr int kGiveThreads = 1024, kGiveCtas = 8;  // one cluster
constexpr int kGiveRound = 4 * kGiveThreads;       // pages that a CTA looks at once
constexpr int kMostRows = 16384;
// Entries of a table that the kernel that gives pages copies itself; more are copied by a
// launch before it.  64 x 128 entries: 8.0 us, with the launch 8.8; 256 x 128: 9.3 and 9.1; 512 x
// 256: 14.0 and 9.7.
constexpr int64_t kFewEntries = 1 << 14;
constexpr int kMoveThreads = 256;
constexpr int kMoveLoads = 4;                      // 16-byte pieces a thread in flight
constexpr int kMoveUnit = 16 * kMoveThreads * kMoveLoads;

// This CTA's shared-memory word in another CTA of the cluster.
__device__ __forceinline__ int peer_int(const int* shared, int rank) {
  uint32_t at;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(shared_address(shared)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// A cluster's barrier in two halves.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int pages_for(int64_t tokens, int log_page) {
  return (int)((tokens + (1ll << log_page) - 1) >> log_page);
}

// Exclusive prefix of one number a thread over the CTA, and the whole sum.
// slots: shared memory for as many numbers as warps.
template <int THREADS>
__device__ __forceinline__ int prefix_of(int v, int* slots, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();  // (the slots' last use)
  if (lane == 31) slots[warp] = s;
  __syncthreads();
  int before = 0;
  sum = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int x = slots[w];
    before += w < warp ? x : 0;
    sum += x;
  }
  return before + s - v;
}

// ---------------------------------------------------------------------------
// The pages' data
// ---------------------------------------------------------------------------
struct PageMove {
  Kv4View from, to;
  int64_t bytes[5];  // of a page in each buffer: codes of K, V, scales of K, V, means
  const int* src;
  const int* dst;
  int n;             // moves,
  const int* count;  // or where the device has their number
  int units;         // pieces of kMoveUnit that a page is cut into
  int unit_of[5];    // the first of each buffer
};

__device__ __forceinline__ uint8_t* buffer_of(const Kv4View& c, int i) {
  return i == 0   ? c.k_codes
         : i == 1 ? c.v_codes
                  : reinterpret_cast<uint8_t*>(i == 2 ? c.k_scales : i == 3 ? c.v_scales : c.k_means);
}

// A CTA a piece of a page.
__device__ __forceinline__ void move_unit(const PageMove& p, int64_t at) {
  const int i = (int)(at / p.units), unit = (int)(at - (int64_t)i * p.units);
  const int from = load(p.src + i), to = load(p.dst + i);
  if (from < 0 || to < 0) return;  // (an entry of no move)
  if (from >= p.from.pages || to >= p.to.pages) {
    if (threadIdx.x == 0) p.from.report(), p.to.report();
    return;
  }
  int b = 0;
#pragma unroll
  for (int k = 1; k < 5; ++k) b += unit >= p.unit_of[k] ? 1 : 0;
  const int64_t bytes = p.bytes[b], first = (int64_t)(unit - p.unit_of[b]) * kMoveUnit;
  const uint8_t* src = buffer_of(p.from, b) + from * bytes;
  uint8_t* dst = buffer_of(p.to, b) + to * bytes;
  uint4 v[kMoveLoads];
#pragma unroll
  for (int k = 0; k < kMoveLoads; ++k) {
    const int64_t o = first + (k * kMoveThreads + threadIdx.x) * 16;
    if (o < bytes) v[k] = load(reinterpret_cast<const uint4*>(src + o));
  }
#pragma unroll
  for (int k = 0; k < kMoveLoads; ++k) {
    const int64_t o = first + (k * kMoveThreads + threadIdx.x) * 16;
    if (o < bytes) *reinterpret_cast<uint4*>(dst + o) = v[k];
  }
}

__global__ void __launch_bounds__(kMoveThreads) kv4_copy_kernel(const PageMove p) {
  wait_for_previous_launch();
  allow_next_launch();
  for (int64_t at = blockIdx.x; at < (int64_t)p.n * p.units; at += gridDim.x) move_unit(p, at);
}

// ---------------------------------------------------------------------------
// The books
// ---------------------------------------------------------------------------
struct BooksParams {
  Kv4View c;
  const int* refs;
  const int* table;
  int64_t table_stride;
  int columns;
  const int* lengths;
  int B;
  const int* parents;  // fork: [n]
  const int* counts;   // reserve: [B], or null: T each
  const int* held;     // release: [B]
  int T, n;
  int copy;            // reserve: what the kernel that gives copies: refs (bit 0), the table (1)
  int* new_table;      // [n][columns], rows new_stride apart
  int64_t new_stride;
  int* new_lengths;
  int* new_refs;
  int* map;            // compact: [pages]
  int* src;            // workspace, fork: [n] the page that row i needs a copy of, or -1
  int* dst;
  int* count;          // compact: the number of moves
};

// new_refs and new_table begin as refs and table (fork: refs; reserve, release: both).
__global__ void __launch_bounds__(kRowsThreads) kv4_books_copy_kernel(const BooksParams p,
                                                                      int with_refs, int with_table) {
  wait_for_previous_launch();
  allow_next_launch();
  const int64_t at = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x;
  const int64_t threads = (int64_t)gridDim.x * kRowsThreads;
  if (with_refs)
    for (int64_t i = at; i < p.c.pages; i += threads) p.new_refs[i] = load(p.refs + i);
  if (!with_table) return;
  for (int64_t i = at; i < (int64_t)p.B * p.columns; i += threads) {
    const int64_t b = i / p.columns, column = i - b * p.columns;
    p.new_table[b * p.new_stride + column] = load(p.table + b * p.table_stride + column);
  }
}

// A CTA a row: what it holds behind its length is given back.  (Launches before it copied
// new_refs and new_table; without a table the entries are the old one's.)
__global__ void __launch_bounds__(kRowsThreads) kv4_release_kernel(const BooksParams p) {
  wait_for_previous_launch();
  allow_next_launch();
  const int b = blockIdx.x;
  const int64_t tokens = max(load(p.lengths + b), 0), most = (int64_t)p.columns << p.c.log_page;
  const int64_t held = max(load(p.held + b), 0);
  if (held > most && threadIdx.x == 0) p.c.report();
  const int first = pages_for(min(tokens, most), p.c.log_page), end = pages_for(min(held, most), p.c.log_page);
  const int* from = p.new_table ? p.new_table + b * p.new_stride : p.table + b * p.table_stride;
  for (int k = first + threadIdx.x; k < end; k += kRowsThreads) {
    const int pg = load(from + k);
    if (pg >= p.c.pages) p.c.report();
    if (pg >= 0 && pg < p.c.pages) atomicAdd(p.new_refs + pg, -1);
    if (p.new_table) p.new_table[b * p.new_stride + k] = -1;
  }
}

// Tokens of old row b, as far as its table goes.
__device__ __forceinline__ int64_t tokens_of(const BooksParams& p, int b) {
  const int64_t n = max(load(p.lengths + b), 0), most = (int64_t)p.columns << p.c.log_page;
  if (n > most && threadIdx.x == 0) p.c.report();
  return min(n, most);
}

// CTAs 0 .. n - 1: the new rows, a CTA each.  The others: the old rows' pages, which
// have as many holders more as the row has children, less its own; a page that is
// not full has one, if there are children.
__global__ void __launch_bounds__(kRowsThreads) kv4_fork_kernel(const BooksParams p) {
  __shared__ int slots[kRowsThreads / 32];
  wait_for_previous_launch();
  allow_next_launch();
  auto parent_of = [&](int i) {
    const int b = load(p.parents + i);
    return b >= p.B ? -1 : b;
  };
  if ((int)blockIdx.x < p.n) {
    const int i = blockIdx.x, parent = parent_of(i);
    if (load(p.parents + i) >= p.B && threadIdx.x == 0) p.c.report();
    int before = 0;  // earlier children of the same parent
    if (parent >= 0)
      for (int k = threadIdx.x; k < i; k += kRowsThreads) before += parent_of(k) == parent ? 1 : 0;
    const bool first = !__syncthreads_or(before);
    const int64_t tokens = parent < 0 ? 0 : tokens_of(p, parent);
    const int pages = pages_for(tokens, p.c.log_page);
    const bool part = (tokens & (p.c.page - 1)) != 0;
    const int* from = p.table + max(parent, 0) * p.table_stride;
    int* to = p.new_table + i * p.new_stride;
    for (int k = threadIdx.x; k < p.columns; k += kRowsThreads) {
      int pg = -1;
      if (k < pages) pg = page_at(p.c, from, p.columns, k);
      const bool copy = part && !first && k == pages - 1;
      if (copy) p.src[i] = pg;
      to[k] = copy ? -1 : pg;
    }
    if (threadIdx.x == 0) {
      if (!(part && !first)) p.src[i] = -1;
      p.new_lengths[i] = parent < 0 ? 0 : max(load(p.lengths + parent), 0);
    }
    return;
  }
  const int b = blockIdx.x - p.n;
  int mine = 0, children = 0;
  for (int k = threadIdx.x; k < p.n; k += kRowsThreads) mine += parent_of(k) == b ? 1 : 0;
  prefix_of<kRowsThreads>(mine, slots, children);
  const int64_t tokens = tokens_of(p, b);
  const int pages = pages_for(tokens, p.c.log_page);
  const bool part = (tokens & (p.c.page - 1)) != 0;
  for (int k = threadIdx.x; k < pages; k += kRowsThreads) {
    const int more = (part && k == pages - 1 ? min(children, 1) : children) - 1;
    const int pg = load(p.table + b * p.table_stride + k);
    if (more != 0 && pg >= 0 && pg < p.c.pages) atomicAdd(p.new_refs + pg, more);
  }
}

// Gives the lowest free pages to the rows that want some, in the order of rows and
// columns: FORK: a copy of one page where src[i] >= 0; else room for the new tokens.
// One cluster: each CTA counts the free pages of its part, and gives those that
// are wanted once it knows how many there are before them.
template <bool FORK>
__global__ void __launch_bounds__(kGiveThreads, 1) kv4_give_kernel(const BooksParams p) {
  extern __shared__ int starts[];  // [n + 1] pages wanted by the rows before
  int* columns = starts + p.n + 1;  // [n] the rows' first new columns
  __shared__ int slots[kGiveThreads / 32];
  __shared__ int mine;
  wait_for_previous_launch();
  allow_next_launch();
  const int tid = threadIdx.x, rank = blockIdx.x;
  // the row's first new column, and how many
  auto wants = [&](int i, int& column) -> int {
    if (FORK) {
      const int64_t tokens =
          min((int64_t)max(load(p.new_lengths + i), 0), (int64_t)p.columns << p.c.log_page);
      column = (int)(tokens >> p.c.log_page);
      return load(p.src + i) >= 0 ? 1 : 0;
    }
    const int64_t tokens = max(load(p.lengths + i), 0);
    const int64_t more = p.counts ? max(load(p.counts + i), 0) : p.T;
    const int64_t all = (tokens + more + p.c.page - 1) >> p.c.log_page;
    const int64_t have = (tokens + p.c.page - 1) >> p.c.log_page;
    column = (int)min(have, (int64_t)p.columns);
    return (int)(min(all, (int64_t)p.columns) - column);
  };
  // this CTA's pages; those of the first round stay in registers, and are asked for before
  // the rows
  const int* refs = !FORK && (p.copy & 1) ? p.refs : p.new_refs;
  const int64_t part = ((int64_t)p.c.pages + kGiveCtas * 4 - 1) / (kGiveCtas * 4) * 4;
  const int64_t begin = min((int64_t)p.c.pages, part * rank), end = min((int64_t)p.c.pages, begin + part);
  const bool whole = (reinterpret_cast<uintptr_t>(refs) & 15u) == 0;
  auto free4 = [&](int64_t page) -> uint32_t {  // of pages page .. page + 3
    uint32_t m = 0;
    if (page + 4 <= end) {
      int4 v;
      if (whole)
        v = load(reinterpret_cast<const int4*>(refs + page));
      else
        v = make_int4(load(refs + page), load(refs + page + 1), load(refs + page + 2), load(refs + page + 3));
      m = (v.x == 0 ? 1u : 0u) | (v.y == 0 ? 2u : 0u) | (v.z == 0 ? 4u : 0u) | (v.w == 0 ? 8u : 0u);
    } else {
      for (int k = 0; k < 4; ++k)
        if (page + k < end && load(refs + page + k) == 0) m |= 1u << k;
    }
    return m;
  };
  const uint32_t first_free = begin + 4 * tid < end ? free4(begin + 4 * tid) : 0u;
  // rows: consecutive ones a thread
  const int per = (p.n + kGiveThreads - 1) / kGiveThreads;
  int sum = 0;
  bool late = false;  // a row whose table is too short
  for (int k = 0; k < per; ++k) {
    const int i = tid * per + k;
    if (i >= p.n) break;
    const int wanted = wants(i, columns[i]);
    starts[i] = wanted;
    sum += wanted;
    if (!FORK) {
      const int64_t all = (int64_t)max(load(p.lengths + i), 0) +
                          (p.counts ? max(load(p.counts + i), 0) : p.T);
      late = late || all > (int64_t)p.columns << p.c.log_page;
    }
  }
  if (late && rank == 0) p.c.report();
  int wanted;
  int at = prefix_of<kGiveThreads>(sum, slots, wanted);
  for (int k = 0; k < per; ++k) {
    const int i = tid * per + k;
    if (i >= p.n) break;
    const int mine = starts[i];
    starts[i] = at;
    at += mine;
  }
  if (tid == 0) starts[p.n] = wanted;
  if (!FORK && (p.copy & 2)) {  // (rows by CTAs; ordered before what is given by the barriers)
    const int64_t entries = (int64_t)p.B * p.columns;
    for (int64_t i = (int64_t)rank * kGiveThreads + tid; i < entries; i += kGiveCtas * kGiveThreads) {
      const int64_t b = i / p.columns, k = i - b * p.columns;
      p.new_table[b * p.new_stride + k] = load(p.table + b * p.table_stride + k);
    }
  }
  int free = __popc(first_free);
  for (int64_t page = begin + 4 * tid + kGiveRound; page < end; page += kGiveRound)
    free += __popc(free4(page));
  if (refs != p.new_refs)
    for (int64_t page = begin + tid; page < end; page += kGiveThreads)
      p.new_refs[page] = load(refs + page);
  int all_free = 0;
  prefix_of<kGiveThreads>(free, slots, all_free);
  if (tid == 0) mine = all_free;
  __syncthreads();
  cluster_barrier();
  int before = 0;
  all_free = 0;
  for (int k = 0; k < kGiveCtas; ++k) {
    const int x = peer_int(&mine, k);
    before += k < rank ? x : 0;
    all_free += x;
  }
  cluster_arrive();  // no CTA leaves while another reads its memory
  auto give = [&](int k, int page) {  // the k-th wanted page
    int lo = 0, hi = p.n;             // last row with starts[row] <= k
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= k) lo = mid; else hi = mid;
    }
    p.new_table[lo * p.new_stride + columns[lo] + (k - starts[lo])] = page;
    if (FORK) p.dst[lo] = page;
    if (page >= 0) p.new_refs[page] = 1;
  };
  // (a round's pages are looked at by all threads before any of them is given)
  for (int64_t first = begin; first < end && before < wanted; first += kGiveRound) {
    const int64_t page = first + 4 * tid;
    uint32_t m = first == begin ? first_free : page < end ? free4(page) : 0u;
    int found;
    int k = before + prefix_of<kGiveThreads>(__popc(m), slots, found);
    before += found;
    for (; m && k < wanted; ++k, m &= m - 1u) give(k, (int)(page + __ffs(m) - 1));
  }
  // what there are no pages for
  if (all_free < wanted) {
    if (tid == 0 && rank == 0) p.c.report();
    for (int k = all_free + rank * kGiveThreads + tid; k < wanted; k += kGiveCtas * kGiveThreads)
      give(k, -1);
  }
  __syncwarp();
  cluster_wait();
}

// Copies of the pages that are not full, as far as they are filled: a CTA a row,
// head and kind (K, V).
__global__ void __launch_bounds__(kMoveThreads) kv4_fork_copy_kernel(const BooksParams p,
                                                                     int code_row, int scale_row) {
  wait_for_previous_launch();
  allow_next_launch();
  const int i = blockIdx.x, h = blockIdx.y;
  const int src = load(p.src + i);
  if (src < 0) return;
  const int dst = load(p.dst + i);
  if (dst < 0) return;
  const int tokens = load(p.new_lengths + i) & (p.c.page - 1);
  const int64_t from = p.c.row(src, h, 0), to = p.c.row(dst, h, 0);
  auto move = [&](uint8_t* buffer, int row) {
    const uint4* a = reinterpret_cast<const uint4*>(buffer + from * row);
    uint4* b = reinterpret_cast<uint4*>(buffer + to * row);
    const int pieces = (tokens * row + 15) / 16;  // (a page holds whole pieces)
    for (int k = threadIdx.x; k < pieces; k += kMoveThreads) {
      const uint4 v = load(a + k);
      const int rest = tokens * row - k * 16;
      if (rest >= 16) {
        b[k] = v;
      } else {  // (the token behind stays as it was)
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int x = 0; x < rest / 4; ++x) reinterpret_cast<uint32_t*>(b + k)[x] = w[x];
      }
    }
  };
  uint8_t* codes = blockIdx.z ? p.c.v_codes : p.c.k_codes;
  move(codes, code_row);
  move(reinterpret_cast<uint8_t*>(blockIdx.z ? p.c.v_scales : p.c.k_scales), scale_row);
}

// The moves that bring the n pages in use to places 0 .. n - 1: those at n and above
// go to the free ones below n, both in ascending order.  One cluster.
__global__ void __launch_bounds__(kGiveThreads, 1) kv4_compact_kernel(const BooksParams p) {
  __shared__ int slots[kGiveThreads / 32];
  __shared__ int mine[3];
  wait_for_previous_launch();
  allow_next_launch();
  const int tid = threadIdx.x, rank = blockIdx.x;
  const int64_t part = ((int64_t)p.c.pages + kGiveCtas - 1) / kGiveCtas;
  const int64_t begin = min((int64_t)p.c.pages, part * rank), end = min((int64_t)p.c.pages, begin + part);
  auto count_used = [&](int64_t from, int64_t to) {
    int used = 0, all;
    for (int64_t page = from + tid; page < to; page += kGiveThreads)
      used += load(p.refs + page) > 0 ? 1 : 0;
    prefix_of<kGiveThreads>(used, slots, all);
    return all;
  };
  const int used = count_used(begin, end);
  if (tid == 0) mine[0] = used;
  __syncthreads();
  cluster_barrier();
  int n = 0;
  for (int k = 0; k < kGiveCtas; ++k) n += peer_int(&mine[0], k);
  // of this CTA's pages: free ones below n, pages in use from n on
  const int64_t border = min(max((int64_t)n, begin), end);
  const int high = count_used(border, end);
  const int low = (int)(border - begin) - (used - high);
  if (tid == 0) mine[1] = low, mine[2] = high;
  __syncthreads();
  cluster_barrier();
  int low_before = 0, high_before = 0, moves = 0;
  for (int k = 0; k < kGiveCtas; ++k) {
    const int a = peer_int(&mine[1], k), b = peer_int(&mine[2], k);
    low_before += k < rank ? a : 0;
    high_before += k < rank ? b : 0;
    moves += b;
  }
  if (tid == 0 && rank == 0) *p.count = moves;
  for (int64_t first = begin; first < end; first += kGiveThreads) {
    const int64_t page = first + tid;
    const bool in_use = page < end && load(p.refs + page) > 0;
    const bool hole = page < end && !in_use && page < n, moving = in_use && page >= n;
    int sum;
    // (both counts in one: fewer than 2^15 of a round)
    const int k = prefix_of<kGiveThreads>((hole ? 1 : 0) | (moving ? 1 << 16 : 0), slots, sum);
    if (hole) p.dst[low_before + (k & 0xFFFF)] = (int)page;
    if (moving) p.src[high_before + (k >> 16)] = (int)page;
    low_before += sum & 0xFFFF;
    high_before += sum >> 16;
    if (page < end) {
      const int holders = load(p.refs + page);
      p.map[page] = in_use ? (int)page : -1;
      if (p.new_refs != p.refs) p.new_refs[page] = holders;
    }
  }
  __threadfence();
  cluster_barrier();
  for (int k = rank * kGiveThreads + tid; k < moves; k += kGiveCtas * kGiveThreads) {
    const int from = __ldcg(p.src + k), to = __ldcg(p.dst + k);
    p.map[from] = to;
    const int holders = load(p.refs + from);
    p.new_refs[to] = holders;
    p.new_refs[from] = 0;
  }
}

// The moves, and the tables by the map.
__global__ void __launch_bounds__(kMoveThreads) kv4_compact_move_kernel(const PageMove m,
                                                                        const BooksParams p) {
  wait_for_previous_launch();
  allow_next_launch();
  for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < (int64_t)p.B * p.columns;
       i += (int64_t)gridDim.x * kMoveThreads) {
    const int64_t b = i / p.columns, column = i - b * p.columns;
    int pg = load(p.table + b * p.table_stride + column);
    if (pg >= p.c.pages) p.c.report();
    if (pg >= 0 && pg < p.c.pages) pg = load(p.map + pg);
    p.new_table[b * p.new_stride + column] = pg;
  }
  const int64_t units = (int64_t)load(m.count) * m.units;
  for (int64_t at = blockIdx.x; at < units; at += gridDim.x) move_unit(m, at);
}

bool ints_ok(const void* p) { return p && !(reinterpret_cast<uintptr_t>(p) & 3u); }

void set_pages(const bsattn_kv4_cache* c, PageMove* m) {
  const int64_t rows = (int64_t)c->kv_heads * c->page_size;
  m->bytes[0] = m->bytes[1] = rows * (c->head_dim / 2);
  m->bytes[2] = m->bytes[3] = rows * (c->head_dim / c->group) * 4;
  m->bytes[4] = (int64_t)c->kv_heads * c->head_dim * 2;
  m->units = 0;
  for (int i = 0; i < 5; ++i) {
    m->unit_of[i] = m->units;
    m->units += (int)((m->bytes[i] + kMoveUnit - 1) / kMoveUnit);
  }
}

// CTAs for so many pieces of pages: as many as run at once, times a few.
int move_grid(int64_t units, int sms) {
  const int64_t most = (int64_t)sms * 32;
  return (int)(units < 1 ? 1 : units < most ? units : most);
}

template <typename Kernel>
cudaError_t launch_cluster(Kernel kernel, size_t smem, cudaStream_t st, const BooksParams& p) {
  return launch_dependent_clusters(kernel, dim3(kGiveCtas), dim3(kGiveThreads), kGiveCtas, smem, st,
                                   p);
}

template <bool FORK>
cudaError_t launch_give(const BooksParams& p, cudaStream_t st) {
  constexpr auto kernel = kv4_give_kernel<FORK>;
  const cudaError_t e = allow_shared_memory<kernel>((2 * kMostRows + 1) * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  return launch_cluster(kernel, (size_t)(2 * p.n + 1) * sizeof(int), st, p);
}

cudaError_t launch_books_copy(const BooksParams& p, bool with_refs, bool with_table, int sms,
                              cudaStream_t st) {
  const int64_t refs = with_refs ? p.c.pages : 0, entries = with_table ? (int64_t)p.B * p.columns : 0;
  const int64_t ctas = (std::max(refs, entries) + kRowsThreads - 1) / kRowsThreads;
  return launch_dependent(kv4_books_copy_kernel, dim3((unsigned)std::min(ctas, (int64_t)sms * 16)),
                          dim3(kRowsThreads), 0, st, p, with_refs ? 1 : 0, with_table ? 1 : 0);
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}
int64_t table_bytes(int64_t rows, int64_t stride, int columns) {
  return ((rows - 1) * stride + columns) * 4;
}

}  // namespace
}  // namespace bsattn

using namespace bsattn;

extern "C" {

bsattn_status bsattn_kv4_copy(const bsattn_kv4_cache* from, const bsattn_kv4_cache* to,
                              const int32_t* src, const int32_t* dst, int n, void* stream) {
  PageMove m{};
  bsattn_status rc = check_cache(from, &m.from);
  if (rc == BSATTN_OK) rc = check_cache(to, &m.to);
  if (rc != BSATTN_OK) return rc;
  if (from->kv_heads != to->kv_heads || from->page_size != to->page_size ||
      from->head_dim != to->head_dim || from->group != to->group)
    return BSATTN_ERR_INVALID_ARG;
  if (!ints_ok(src) || !ints_ok(dst) || n <= 0) return BSATTN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  set_pages(from, &m);
  m.src = src;
  m.dst = dst;
  m.n = n;
  return from_cuda(launch_dependent(kv4_copy_kernel,
                                    dim3(move_grid((int64_t)n * m.units, device_sm_count(dev))),
                                    dim3(kMoveThreads), 0, static_cast<cudaStream_t>(stream), m));
}

size_t bsattn_kv4_fork_workspace(int n) { return n > 0 ? (size_t)n * 2 * sizeof(int) : 0; }

bsattn_status bsattn_kv4_fork(const bsattn_kv4_cache* cache, const int32_t* refs,
                              const int32_t* block_table, int64_t table_stride, int columns,
                              const int32_t* lengths, int B, const int32_t* parents, int n,
                              int32_t* new_table, int32_t* new_lengths, int32_t* new_refs,
                              void* workspace, size_t workspace_bytes, void* stream) {
  BooksParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!ints_ok(refs) || !ints_ok(block_table) || !ints_ok(lengths) || !ints_ok(parents) ||
      !ints_ok(new_table) || !ints_ok(new_lengths) || !ints_ok(new_refs) || !aligned16(new_refs))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || n <= 0 || columns <= 0 || table_stride < 0) return BSATTN_ERR_INVALID_ARG;
  if (B > kMostRows || n > kMostRows || cache->kv_heads > 65535) return BSATTN_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) || workspace_bytes < bsattn_kv4_fork_workspace(n))
    return BSATTN_ERR_INVALID_ARG;
  // the old rows are read while the new ones are written
  if (overlap(new_table, (int64_t)n * columns * 4, block_table,
              table_bytes(B, table_stride, columns)) ||
      overlap(new_lengths, (int64_t)n * 4, lengths, (int64_t)B * 4) ||
      overlap(new_lengths, (int64_t)n * 4, parents, (int64_t)n * 4) ||
      overlap(new_table, (int64_t)n * columns * 4, parents, (int64_t)n * 4) ||
      (new_refs != refs &&
       overlap(new_refs, (int64_t)cache->pages * 4, refs, (int64_t)cache->pages * 4)))
    return BSATTN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  p.refs = refs;
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.B = B;
  p.parents = parents;
  p.n = n;
  p.new_table = new_table;
  p.new_stride = columns;
  p.new_lengths = new_lengths;
  p.new_refs = new_refs;
  p.src = static_cast<int*>(workspace);
  p.dst = p.src + n;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (new_refs != refs) e = launch_books_copy(p, true, false, device_sm_count(dev), st);
  if (e == cudaSuccess)
    e = launch_dependent(kv4_fork_kernel, dim3(n + B), dim3(kRowsThreads), 0, st, p);
  if (e == cudaSuccess) e = launch_give<true>(p, st);
  if (e == cudaSuccess)
    e = launch_dependent(kv4_fork_copy_kernel, dim3(n, cache->kv_heads, 2), dim3(kMoveThreads), 0,
                         st, p, cache->head_dim / 2, cache->head_dim / cache->group * 4);
  return from_cuda(e);
}

bsattn_status bsattn_kv4_reserve(const bsattn_kv4_cache* cache, const int32_t* refs,
                                 const int32_t* block_table, int64_t table_stride, int columns,
                                 const int32_t* lengths, const int32_t* counts, int T, int B,
                                 int32_t* new_table, int64_t new_stride, int32_t* new_refs,
                                 void* stream) {
  BooksParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!ints_ok(refs) || !ints_ok(block_table) || !ints_ok(lengths) ||
      (counts && !ints_ok(counts)) || !ints_ok(new_table) || !ints_ok(new_refs) ||
      !aligned16(new_refs))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || columns <= 0 || T < 0 || table_stride < 0 || (B > 1 && new_stride < columns))
    return BSATTN_ERR_INVALID_ARG;
  if (B > kMostRows) return BSATTN_ERR_UNSUPPORTED;
  const bool same = new_table == block_table && (new_stride == table_stride || B == 1);
  if ((!same && overlap(new_table, table_bytes(B, new_stride, columns), block_table,
                        table_bytes(B, table_stride, columns))) ||
      (new_refs != refs &&
       overlap(new_refs, (int64_t)cache->pages * 4, refs, (int64_t)cache->pages * 4)))
    return BSATTN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  p.refs = refs;
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.counts = counts;
  p.T = T;
  p.B = p.n = B;
  p.new_table = new_table;
  p.new_stride = new_stride;
  p.new_refs = new_refs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (same || (int64_t)B * columns <= kFewEntries)
    p.copy = (same ? 0 : 2) | (new_refs != refs ? 1 : 0);
  else
    e = launch_books_copy(p, new_refs != refs, true, device_sm_count(dev), st);
  if (e == cudaSuccess) e = launch_give<false>(p, st);
  return from_cuda(e);
}

bsattn_status bsattn_kv4_release(const bsattn_kv4_cache* cache, const int32_t* refs,
                                 const int32_t* block_table, int64_t table_stride, int columns,
                                 const int32_t* lengths, const int32_t* held, int B,
                                 int32_t* new_table, int64_t new_stride, int32_t* new_refs,
                                 void* stream) {
  BooksParams p{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!ints_ok(refs) || !ints_ok(block_table) || !ints_ok(lengths) || !ints_ok(held) ||
      (new_table && !ints_ok(new_table)) || !ints_ok(new_refs) || !aligned16(new_refs))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || columns <= 0 || table_stride < 0 || (new_table && B > 1 && new_stride < columns))
    return BSATTN_ERR_INVALID_ARG;
  if (B > kMostRows) return BSATTN_ERR_UNSUPPORTED;
  const bool same = !new_table || (new_table == block_table && (new_stride == table_stride || B == 1));
  if ((!same && overlap(new_table, table_bytes(B, new_stride, columns), block_table,
                        table_bytes(B, table_stride, columns))) ||
      (new_refs != refs &&
       overlap(new_refs, (int64_t)cache->pages * 4, refs, (int64_t)cache->pages * 4)))
    return BSATTN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  p.refs = refs;
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.lengths = lengths;
  p.held = held;
  p.B = B;
  p.new_table = new_table;
  p.new_stride = new_stride;
  p.new_refs = new_refs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (!same || new_refs != refs) e = launch_books_copy(p, new_refs != refs, !same, device_sm_count(dev), st);
  if (e == cudaSuccess) e = launch_dependent(kv4_release_kernel, dim3(B), dim3(kRowsThreads), 0, st, p);
  return from_cuda(e);
}

size_t bsattn_kv4_compact_workspace(int pages) {
  return pages > 0 ? (size_t)(2 * (int64_t)pages + 4) * sizeof(int) : 0;
}

bsattn_status bsattn_kv4_compact(const bsattn_kv4_cache* cache, const int32_t* refs,
                                 const int32_t* block_table, int64_t table_stride, int columns,
                                 int B, int32_t* new_table, int64_t new_stride, int32_t* new_refs,
                                 int32_t* page_map, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  BooksParams p{};
  PageMove m{};
  const bsattn_status rc = check_cache(cache, &p.c);
  if (rc != BSATTN_OK) return rc;
  if (!ints_ok(refs) || !ints_ok(block_table) || !ints_ok(new_table) || !ints_ok(new_refs) ||
      !ints_ok(page_map))
    return BSATTN_ERR_INVALID_ARG;
  if (B <= 0 || columns <= 0 || table_stride < 0 || (B > 1 && new_stride < columns))
    return BSATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < bsattn_kv4_compact_workspace(cache->pages))
    return BSATTN_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)cache->pages * 4;
  const bool same = new_table == block_table && (new_stride == table_stride || B == 1);
  if ((!same && overlap(new_table, table_bytes(B, new_stride, columns), block_table,
                        table_bytes(B, table_stride, columns))) ||
      (new_refs != refs && overlap(new_refs, bytes, refs, bytes)) ||
      overlap(page_map, bytes, refs, bytes) || overlap(page_map, bytes, new_refs, bytes))
    return BSATTN_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSATTN_ERR_CUDA;
  const int sms = device_sm_count(dev);
  p.refs = refs;
  p.table = block_table;
  p.table_stride = table_stride;
  p.columns = columns;
  p.B = B;
  p.new_table = new_table;
  p.new_stride = new_stride;
  p.new_refs = new_refs;
  p.map = page_map;
  p.count = static_cast<int*>(workspace);
  p.src = p.count + 4;
  p.dst = p.src + cache->pages;
  m.from = m.to = p.c;
  set_pages(cache, &m);
  m.src = p.src;
  m.dst = p.dst;
  m.count = p.count;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  e = launch_cluster(kv4_compact_kernel, 0, st, p);
  // (at most half of the pages move)
  if (e == cudaSuccess)
    e = launch_dependent(kv4_compact_move_kernel,
                         dim3(move_grid(((int64_t)cache->pages + 1) / 2 * m.units, sms)),
                         dim3(kMoveThreads), 0, st, m, p);
  return from_cuda(e);
}

}  // extern "C"
