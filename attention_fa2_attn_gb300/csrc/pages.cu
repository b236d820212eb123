// pages.cu -- the pages of a cache that several sequences share: forking a sequence, copying
// pages, giving back those that nobody holds any more, and moving the live ones together.
//
// What is kept. Row b of the block table holds the ceil(seqlens[b] / 16) pages of sequence b.
// shares[p] is how many sequences hold page p beside its first owner, so a page that
// fa_paged_plan hands out starts at 0 and needs no call of its own.
//
// fa_pages_fork. Child i gets the whole pages of its parent (shares + 1 each) and, where the
// parent's last page is not full, a page of its own from the free list, in the order of i.
// One launch without any exchange between blocks: a warp takes a child, and of the blocks that
// write a row (128 entries each) the first counts by itself how many of the children before it
// need a page. That is work that grows with the square of their number, so it is limited. Bound
// by launch and by two round trips to L2 (parent -> length -> table row); in a graph 16 children
// of tables of 64 pages 2.5 us, 1024 of 512 pages 3.6, 16384 of 1024 75, 65536 of 2048 751 (2034
// where every block of a row counted).
//
// fa_pages_copy. Bound by HBM: every copied byte is read once and written once. A warp moves
// 8 KB of a page at a time, sixteen 16-byte vectors a lane in flight (1.07 GB read and written:
// 163 us, 6.6 TB/s; 167 us with eight, 172 with four).
//
// fa_pages_free, fa_pages_compact. Both need sets of pages in ascending order, so that the
// lists they give do not depend on which atomic came first: a bit for each page of the pool.
// One launch of one cluster of CTAs: each CTA keeps the bits of its part of the pool in shared
// memory, all of them set bits there from their entries of the table, and cluster barriers
// stand where three or five launches would.
//   free: shares[p] is counted down for each of the entries; who finds it at 0 already sets
//   p's bit. Bits in order are the freed list. An SM does one count in about two cycles, so
//   many entries are counted down by the whole GPU first, which leaves -1 where nobody holds a
//   page any more, and the cluster takes its bits from there: three launches (256 of 512 rows,
//   164 000 entries, 524 000 pages: one cluster alone 32 us). Counts that meet on few addresses
//   are no slower (512 rows of 640 pages: 20.3 us where all hold the same 600, 20.0 where none
//   holds another's).
//   compact: a bit for each live page. With n live pages from `first` on, they end up in
//   [first, first + n): a live page behind that moves into a hole before it, the i-th of
//   these into the i-th of those. Sources and holes are apart, so the copies need no order.
//   A page's place in either list is the number of bits before it, from sums over the words.
#include <atomic>
#include <initializer_list>

#include "launch.cuh"

namespace fa {

constexpr int kPgTokens = 16;

// Pages of sequence b in its row, from a length clamped to what the row holds.
__device__ __forceinline__ int pg_len(int s, int max_pages, bool& clamped) {
  const int n = max(0, min(s, max_pages * kPgTokens));
  clamped |= n != s;
  return n;
}
__device__ __forceinline__ int pg_pages(int tokens) { return (tokens + kPgTokens - 1) / kPgTokens; }

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------
constexpr int kForkWarps = 8;   // children of a block
constexpr int kForkRows = 4;    // entries of a lane, in flight together
constexpr int kForkChunk = kForkRows * 32;

struct ForkParams {
  const int* table;
  const int* seqlens;
  const int* parents;
  const int* free_pages;
  int* shares;
  int* table_out;
  int* lens_out;
  int* src;
  int* dst;
  int* used;
  int B, n, max_pages, num_free, num_pages;
  unsigned* err;
};

__device__ __forceinline__ int fork_len(const ForkParams& p, int parent, bool& bad) {
  if (parent < 0 || parent >= p.B) {
    bad |= parent != -1;
    return 0;
  }
  return pg_len(__ldg(p.seqlens + parent), p.max_pages, bad);
}

__global__ void __launch_bounds__(kForkWarps * 32) pages_fork_kernel(const ForkParams p) {
  __shared__ int partial[kForkWarps];
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i0 = blockIdx.x * kForkWarps, i = i0 + warp;
  // The block of a row's first entries alone counts, and writes the child's last page wherever that
  // is. What it counts first is on its way with this child's parent, length and row.
  const bool first = blockIdx.y == 0;
  const int parent = i < p.n ? __ldg(p.parents + i) : -1;
  const int far = first && static_cast<int>(threadIdx.x) < i0 ? __ldg(p.parents + threadIdx.x) : -1;
  const int near = first && lane < warp && i0 + lane < p.n ? __ldg(p.parents + i0 + lane) : -1;
  bool bad = false, ignored = false;
  const int len = fork_len(p, parent, bad);
  int sum = fork_len(p, far, ignored) % kPgTokens != 0;
  const int beside = fork_len(p, near, ignored) % kPgTokens != 0;
  const int full = len / kPgTokens, part = len % kPgTokens != 0;
  const int* row = p.table + static_cast<size_t>(parent >= 0 && parent < p.B ? parent : 0) * p.max_pages;
  const int j0 = blockIdx.y * kForkChunk + lane;
  int e[kForkRows];
#pragma unroll
  for (int k = 0; k < kForkRows; ++k) {
    const int j = j0 + 32 * k;
    e[k] = i < p.n && j < full ? __ldg(row + j) : 0;
  }
  const int copied = first && part ? __ldg(row + full) : -1;
  int before = 0;
  if (first) {
#pragma unroll 4
    for (int c = threadIdx.x + kForkWarps * 32; c < i0; c += kForkWarps * 32)
      sum += fork_len(p, __ldg(p.parents + c), ignored) % kPgTokens != 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) partial[warp] = sum;
    __syncthreads();
    before = beside + (lane < kForkWarps ? partial[lane] : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (i >= p.n) return;
  int* out = p.table_out + static_cast<size_t>(i) * p.max_pages;
#pragma unroll
  for (int k = 0; k < kForkRows; ++k) {
    const int j = j0 + 32 * k;
    if (j >= p.max_pages || (part && j == full)) continue;
    if (j < full) {
      if (e[k] >= 0 && e[k] < p.num_pages) atomicAdd(p.shares + e[k], 1); else bad = true;
    }
    out[j] = e[k];
  }
  if (first && lane == 0) {
    int from = -1, to = -1;
    if (part) {
      int fresh = before < p.num_free ? __ldg(p.free_pages + before) : -1;
      if (fresh < 0 || fresh >= p.num_pages) fresh = -1;
      const bool there = copied >= 0 && copied < p.num_pages;
      bad |= fresh < 0 || !there;
      if (fresh >= 0 && there) {
        from = copied;
        to = fresh;
      }
      out[full] = fresh;
    }
    p.src[i] = from;
    p.dst[i] = to;
    p.lens_out[i] = len;
    if (i == p.n - 1) *p.used = before + part;
  }
  if (bad) record_error(p.err, FA_ERR_BOUNDS, SITE_PAGES_FORK);
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------
constexpr int kCopyVecs = 16;  // 16-byte vectors of a lane in flight
constexpr int kCopyThreads = 256;

struct CopyParams {
  uint4* pool[2];
  const int* src;
  const int* dst;
  const int* count;       // may be null
  int n, num_pages;
  unsigned parts;         // 8 KB parts of a page
  long long page_vecs;    // 16-byte vectors of a page
  long long layer_vecs;   // and of a layer
  int sides;              // layers * 2
  unsigned* err;
};

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyParams p) {
  pdl_wait();
  pdl_launch();
  const int lane = threadIdx.x & 31;
  const unsigned warps = gridDim.x * (kCopyThreads / 32);
  const unsigned warp = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
  const int n = p.count ? max(0, min(p.n, __ldg(p.count))) : p.n;
  // (pair, layer and pool, part), the parts of a page side by side
  const unsigned long long per = static_cast<unsigned long long>(p.sides) * p.parts, total = per * n;
  for (unsigned long long at = warp; at < total; at += warps) {
    const unsigned long long pair = at / per;
    const unsigned rest = static_cast<unsigned>(at - pair * per);
    const unsigned side = rest / p.parts, part = rest - side * p.parts;
    const int a = __ldg(p.src + pair), b = __ldg(p.dst + pair);
    if (a == -1 || b == -1) continue;
    if (a < 0 || a >= p.num_pages || b < 0 || b >= p.num_pages) {
      if (lane == 0) record_error(p.err, FA_ERR_BOUNDS, SITE_PAGES_COPY);
      continue;
    }
    uint4* layer = p.pool[side & 1] + (side >> 1) * p.layer_vecs;
    const long long first = static_cast<long long>(part) * (32 * kCopyVecs) + lane;
    const uint4* from = layer + a * p.page_vecs;
    uint4* to = layer + b * p.page_vecs;
    uint4 v[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (first + 32 * k < p.page_vecs) v[k] = __ldcs(from + first + 32 * k);
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k)
      if (first + 32 * k < p.page_vecs) __stcs(to + first + 32 * k, v[k]);
  }
}

// ---------------------------------------------------------------------------
// free and compact: one cluster
// ---------------------------------------------------------------------------
constexpr int kSetThreads = 1024;
constexpr int kSetMaxCluster = 16;

struct SetParams {
  const int* table;
  const int* seqlens;
  const int* rows;    // free: may be null, all rows
  const int* shares;
  int* shares_out;
  int* table_out;     // compact
  int* list0;         // free: the freed pages; compact: sources
  int* list1;         // compact: destinations
  int* counts;        // free: [1]; compact: [2] moves, live pages
  int B, n;           // n: rows to go over
  int max_pages, num_pages, first;
  long long cap;      // entries of the lists
  int words;          // 32-page words of a CTA's part
  int C;
  unsigned* err;
};

__device__ __forceinline__ void set_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// The place of this CTA's shared memory at `p` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t set_in_cta(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t set_ld(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void set_or(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

constexpr int kSetRows = 4;  // chunks of 32 entries of a warp, in flight together

// Calls f(row of the table, place in it, entry, whether the row's sequence holds it) for the
// entries of the rows; those behind a sequence's pages only with ALL (the compact call copies
// them).
template <bool ALL, int THREADS = kSetThreads, typename F>
__device__ __forceinline__ void set_entries(const SetParams& p, bool& bad, const F& f) {
  const int lane = threadIdx.x & 31;
  const unsigned chunks = (p.max_pages + 31) / 32;
  const unsigned long long items = static_cast<unsigned long long>(p.n) * chunks;
  const unsigned warps = gridDim.x * (THREADS / 32);
  const unsigned warp = blockIdx.x * (THREADS / 32) + (threadIdx.x >> 5);
  for (unsigned long long at = warp; at < items; at += static_cast<unsigned long long>(warps) * kSetRows) {
    int row[kSetRows], j[kSetRows], pages[kSetRows], e[kSetRows];
#pragma unroll
    for (int k = 0; k < kSetRows; ++k) {
      const unsigned long long it = at + static_cast<unsigned long long>(warps) * k;
      row[k] = -1;
      j[k] = pages[k] = 0;
      if (it >= items) continue;
      const unsigned r = static_cast<unsigned>(it / chunks);
      j[k] = static_cast<int>((static_cast<unsigned>(it - static_cast<unsigned long long>(r) * chunks)) * 32 + lane);
      row[k] = p.rows ? __ldg(p.rows + r) : static_cast<int>(r);
    }
#pragma unroll
    for (int k = 0; k < kSetRows; ++k) {
      if (row[k] < 0 || row[k] >= p.B) {
        bad |= row[k] != -1;
        row[k] = -1;
        continue;
      }
      pages[k] = pg_pages(pg_len(__ldg(p.seqlens + row[k]), p.max_pages, bad));
    }
#pragma unroll
    for (int k = 0; k < kSetRows; ++k) {
      e[k] = -1;
      if (row[k] >= 0 && j[k] < (ALL ? p.max_pages : pages[k]))
        e[k] = p.table[static_cast<size_t>(row[k]) * p.max_pages + j[k]];
    }
#pragma unroll
    for (int k = 0; k < kSetRows; ++k)
      if (row[k] >= 0 && j[k] < (ALL ? p.max_pages : pages[k])) f(row[k], j[k], e[k], j[k] < pages[k]);
  }
}

// MODE 0: free; 1: compact; 2: free, the entries counted down already.
template <int MODE>
__global__ void __launch_bounds__(kSetThreads, 1) pages_set_kernel(const SetParams p) {
  constexpr bool COMPACT = MODE == 1;
  extern __shared__ uint32_t set_smem[];
  uint32_t* bits = set_smem;              // [words]: this CTA's part of the pool
  uint32_t* pre = set_smem + p.words;     // [words]: bits of the part before each word
  __shared__ int warp_sum[32];
  __shared__ int part_bits;               // this part's
  __shared__ int base_of[kSetMaxCluster + 1];  // bits of the parts before each
  __shared__ int low;                     // compact: live pages that stay
  const int rank = static_cast<int>(blockIdx.x), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int part_pages = p.words * 32;
  const int page0 = rank * part_pages;    // (a pool has at most 2^22 pages)
  pdl_wait();
  pdl_launch();
  bool bad = false;

  if constexpr (MODE == 2) {
    constexpr int IN = 4;  // words of a warp in flight
    for (int w = warp; w < p.words; w += IN * (kSetThreads / 32)) {
      int left[IN];
#pragma unroll
      for (int k = 0; k < IN; ++k) {
        const int x = w + k * (kSetThreads / 32), page = page0 + x * 32 + lane;
        left[k] = x < p.words && page < p.num_pages ? p.shares_out[page] : 0;
      }
#pragma unroll
      for (int k = 0; k < IN; ++k) {
        const unsigned v = __ballot_sync(0xffffffffu, left[k] < 0);
        if (lane == 0 && w + k * (kSetThreads / 32) < p.words) bits[w + k * (kSetThreads / 32)] = v;
      }
    }
    __syncthreads();
  } else {
  for (int w = tid; w < p.words; w += kSetThreads) bits[w] = 0u;
  if (!COMPACT && p.shares_out != p.shares) {
    const int last = min(p.num_pages, page0 + part_pages);
#pragma unroll 4
    for (int x = page0 + tid; x < last; x += kSetThreads) p.shares_out[x] = __ldg(p.shares + x);
  }
  set_cluster_sync();

  auto mark = [&](int page) {
    const int owner = page / part_pages, at = page - owner * part_pages;
    set_or(set_in_cta(bits + (at >> 5), owner), 1u << (at & 31));
  };
  set_entries<false>(p, bad, [&](int, int, int e, bool) {
    if (e < 0 || e >= p.num_pages) {
      bad = true;
      return;
    }
    if (COMPACT) {
      if (e >= p.first) mark(e);
    } else {
      const int left = atomicSub(p.shares_out + e, 1);
      if (left == 0) mark(e);       // nobody else holds it
      else bad |= left < 0;         // given back more often than it is held
    }
  });
  if (bad) record_error(p.err, FA_ERR_BOUNDS, COMPACT ? SITE_PAGES_COMPACT : SITE_PAGES_FREE);
  set_cluster_sync();
  }

  // bits before each word, of the part and of the parts before it
  {
    const int per = (p.words + kSetThreads - 1) / kSetThreads;
    const int lo = min(p.words, tid * per), hi = min(p.words, lo + per);
    int mine = 0;
    for (int w = lo; w < hi; ++w) mine += __popc(bits[w]);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int sums = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, sums, o);
      if (lane >= o) sums += y;
    }
    int at = inc - mine + (warp ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0);
    for (int w = lo; w < hi; ++w) {
      pre[w] = at;
      at += __popc(bits[w]);
    }
    if (tid == 31) part_bits = sums;
  }
  set_cluster_sync();
  if (warp == 0) {
    int v = lane < p.C ? static_cast<int>(set_ld(set_in_cta(&part_bits, lane))) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane == 0) base_of[0] = 0;
    if (lane < p.C) base_of[lane + 1] = v;
  }
  __syncthreads();
  const int all = base_of[p.C], base = base_of[rank];

  if constexpr (!COMPACT) {
    for (int w = warp; w < p.words; w += kSetThreads / 32) {
      const uint32_t v = bits[w];
      if ((v >> lane) & 1u) {
        const int page = page0 + w * 32 + lane;
        const int at = base + static_cast<int>(pre[w]) + __popc(v & ((1u << lane) - 1u));
        if (at < p.cap) p.list0[at] = page;  // (as many as were given back, unless shares were negative)
        p.shares_out[page] = 0;
      }
    }
    if (MODE == 0)
      for (long long x = all + static_cast<long long>(rank) * kSetThreads + tid; x < p.cap; x += static_cast<long long>(p.C) * kSetThreads)
        p.list0[x] = -1;
    if (rank == 0 && tid == 0) {
      p.counts[0] = static_cast<int>(min(static_cast<long long>(all), p.cap));
      if (all > p.cap) record_error(p.err, FA_ERR_BOUNDS, SITE_PAGES_FREE);
    }
  } else {
    // live pages before page x
    auto rank_of = [&](int x) -> int {
      const int owner = x / part_pages, at = x - owner * part_pages;
      if (owner >= p.C) return all;
      const uint32_t v = set_ld(set_in_cta(bits + (at >> 5), owner)), b = set_ld(set_in_cta(pre + (at >> 5), owner));
      return base_of[owner] + static_cast<int>(b) + __popc(v & ((1u << (at & 31)) - 1u));
    };
    const int end = p.first + all;  // (at most num_pages)
    if (tid == 0) low = rank_of(end);
    __syncthreads();
    const int stay = low, moves = all - stay;
    for (int w = warp; w < p.words; w += kSetThreads / 32) {
      const int page = page0 + w * 32 + lane;
      if (page >= p.num_pages) continue;
      const uint32_t v = bits[w];
      const bool live = (v >> lane) & 1u;
      const int at = base + static_cast<int>(pre[w]) + __popc(v & ((1u << lane) - 1u));
      if (page < p.first) {
        p.shares_out[page] = p.shares[page];
      } else if (live && page >= end) {
        p.list0[at - stay] = page;
      } else {
        if (!live && page < end) p.list1[page - p.first - at] = page;
        p.shares_out[page] = live ? p.shares[page] : 0;
      }
    }
    for (long long x = moves + static_cast<long long>(rank) * kSetThreads + tid; x < p.cap; x += static_cast<long long>(p.C) * kSetThreads)
      p.list0[x] = p.list1[x] = -1;
    if (rank == 0 && tid == 0) {
      p.counts[0] = moves;
      p.counts[1] = all;
    }
    set_cluster_sync();  // the destinations are there
    for (int w = warp; w < p.words; w += kSetThreads / 32) {
      const int page = page0 + w * 32 + lane;
      const uint32_t v = bits[w];
      if (page >= end && ((v >> lane) & 1u)) {
        const int at = base + static_cast<int>(pre[w]) + __popc(v & ((1u << lane) - 1u));
        const int s = p.shares[page];
        p.shares_out[__ldcg(p.list1 + at - stay)] = s;
        p.shares_out[page] = 0;
      }
    }
    bool ignored = false;
    set_entries<true>(p, ignored, [&](int row, int j, int e, bool live) {
      if (live && e >= end && e < p.num_pages) e = __ldcg(p.list1 + rank_of(e) - stay);
      p.table_out[static_cast<size_t>(row) * p.max_pages + j] = e;
    });
  }
  set_cluster_sync();  // nobody leaves while others read its shared memory
}

// What the whole GPU does of a large free: the copy of the shares and the list's -1, then the
// counts.
constexpr int kFreeThreads = 256;
__global__ void __launch_bounds__(kFreeThreads) pages_free_begin_kernel(const SetParams p) {
  pdl_wait();
  pdl_launch();
  const long long at = static_cast<long long>(blockIdx.x) * kFreeThreads + threadIdx.x, step = static_cast<long long>(gridDim.x) * kFreeThreads;
  if (p.shares_out != p.shares)
    for (long long x = at; x < p.num_pages; x += step) p.shares_out[x] = __ldg(p.shares + x);
  for (long long x = at; x < p.cap; x += step) p.list0[x] = -1;
}
__global__ void __launch_bounds__(kFreeThreads) pages_free_count_kernel(const SetParams p) {
  pdl_wait();
  pdl_launch();
  bool bad = false;
  set_entries<false, kFreeThreads>(p, bad, [&](int, int, int e, bool) {
    if (e < 0 || e >= p.num_pages)
      bad = true;
    else
      bad |= atomicSub(p.shares_out + e, 1) < 0;
  });
  if (bad) record_error(p.err, FA_ERR_BOUNDS, SITE_PAGES_FREE);
}
// Entries from which on that is done: one cluster / three launches, us: 64 000 entries 14.1 / 16.9,
// 262 144 entries 32.1 / 18.5, 524 288 entries 51.4 / 19.6.
constexpr long long kFreeLarge = 131072;

// CTAs of the cluster. A cluster's barriers cost a microsecond that a few chunks of 32 entries do
// not make up for; many are done faster by more SMs (compact, us, 1 / 4 / 16 CTAs: 16 chunks 6.2 /
// 7.7 / 7.2, 128 chunks 11.3 / 9.2 / 8.7, 512 chunks 31.8 / 16.6 / 11.8; free: 32 chunks 5.7 / 6.7 /
// 6.5, 256 chunks 13.4 / 9.3 / 7.5).
static int set_cluster(long long rows, int max_pages, int num_pages) {
  const long long chunks = rows * ((max_pages + 31) / 32);
  if (chunks > 128 || num_pages > 32768) return kSetMaxCluster;
  return chunks > 32 ? 8 : 1;
}

template <int MODE>
static int launch_set(SetParams& p, cudaStream_t stream) {
  p.C = set_cluster(MODE == 2 ? 0 : p.n, p.max_pages, p.num_pages);
  p.words = (p.num_pages + 32 * p.C - 1) / (32 * p.C);
  const size_t smem = static_cast<size_t>(p.words) * 8;
  auto kfn = pages_set_kernel<MODE>;
  // the attributes hold for the life of the device's context: asked for once per device
  static std::atomic<unsigned long long> asked{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda_failure(e);
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, FA_PAGES_MAX / 32 / kSetMaxCluster * 8);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kfn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return record_cuda_failure(e);
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_dependent_cluster(kfn, dim3(p.C), p.C, dim3(kSetThreads), smem, stream, p);
}

static bool pg_off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

struct PgRange {
  const void* p;
  long long bytes;
};
// Whether one of the outputs shares a byte with an input or another output.
static bool pg_meet(std::initializer_list<PgRange> outs, std::initializer_list<PgRange> ins) {
  for (const PgRange* o = outs.begin(); o != outs.end(); ++o) {
    for (const PgRange& x : ins)
      if (overlap(o->p, o->bytes, x.p, x.bytes)) return true;
    for (const PgRange* x = outs.begin(); x != o; ++x)
      if (overlap(o->p, o->bytes, x->p, x->bytes)) return true;
  }
  return false;
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_pages_fork(const int* block_table, const int* seqlens, const int* parents, const int* free_pages,
                        int num_free, int* shares, int* table_out, int* lens_out, int* copy_src, int* copy_dst,
                        int* pages_used, int B, int n, int max_pages, int page_size, int num_pages, void* stream) {
  if (B < 1 || n < 1 || max_pages < 1 || num_pages < 1 || num_free < 0) return FA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(seqlens),
                        static_cast<const void*>(parents), static_cast<const void*>(shares),
                        static_cast<const void*>(table_out), static_cast<const void*>(lens_out),
                        static_cast<const void*>(copy_src), static_cast<const void*>(copy_dst),
                        static_cast<const void*>(pages_used)})
    if (!x || pg_off(x, 4)) return FA_ERR_INVALID_ARG;
  if ((num_free > 0 && !free_pages) || pg_off(free_pages, 4)) return FA_ERR_INVALID_ARG;
  if (page_size != kPgTokens) return FA_ERR_UNSUPPORTED;
  const long long mp = max_pages;
  if (mp * kPgTokens >= (1ll << 31) || mp * B >= (1ll << 31) || mp * n >= (1ll << 31) ||
      num_pages * 16ll >= (1ll << 31) || mp > 65535ll * kForkChunk || n > FA_FORK_MAX)
    return FA_ERR_UNSUPPORTED;
  if (pg_meet({{table_out, 4 * mp * n}, {lens_out, 4ll * n}, {copy_src, 4ll * n}, {copy_dst, 4ll * n}, {pages_used, 4},
               {shares, 4ll * num_pages}},
              {{block_table, 4 * mp * B}, {seqlens, 4ll * B}, {parents, 4ll * n}, {free_pages, 4ll * num_free}}))
    return FA_ERR_INVALID_ARG;
  ForkParams p = {block_table, seqlens, parents, free_pages, shares, table_out, lens_out, copy_src, copy_dst,
                  pages_used, B, n, max_pages, num_free, num_pages, device_error_word()};
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  const dim3 grid((n + kForkWarps - 1) / kForkWarps, (max_pages + kForkChunk - 1) / kForkChunk);
  return static_cast<fa_status>(
      launch_dependent(pages_fork_kernel, grid, dim3(kForkWarps * 32), 0, static_cast<cudaStream_t>(stream), p));
}

fa_status fa_pages_copy(void* k_pages, void* v_pages, const int* src, const int* dst, const int* count, int n,
                        int layers, int num_pages, int page_size, int Hkv, int d, void* stream) {
  if (!k_pages || !v_pages || !src || !dst) return FA_ERR_INVALID_ARG;
  if (pg_off(k_pages, 16) || pg_off(v_pages, 16) || pg_off(src, 4) || pg_off(dst, 4) || pg_off(count, 4))
    return FA_ERR_INVALID_ARG;
  if (n < 1 || layers < 1 || num_pages < 1 || Hkv < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (page_size != kPgTokens || num_pages * 16ll >= (1ll << 31) || layers > (1 << 20) || Hkv > 65535 || d > 1024)
    return FA_ERR_UNSUPPORTED;
  const long long page = 2ll * kPgTokens * Hkv * d;  // bytes, a multiple of 32
  const long long layer = page * num_pages;          // at most 2^58
  if (layer > (1ll << 60) / layers) return FA_ERR_UNSUPPORTED;
  const long long pool = layer * layers, ints = 4ll * n;
  if (pg_meet({{k_pages, pool}, {v_pages, pool}}, {{src, ints}, {dst, ints}, {count, 4}})) return FA_ERR_INVALID_ARG;
  CopyParams p = {};
  p.pool[0] = static_cast<uint4*>(k_pages);
  p.pool[1] = static_cast<uint4*>(v_pages);
  p.src = src;
  p.dst = dst;
  p.count = count;
  p.n = n;
  p.num_pages = num_pages;
  p.page_vecs = page / 16;
  p.layer_vecs = layer / 16;
  p.parts = static_cast<unsigned>((p.page_vecs + 32 * kCopyVecs - 1) / (32 * kCopyVecs));
  p.sides = 2 * layers;
  p.err = device_error_word();
  const int sms = device_sm_count();
  if (!p.err || !sms) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  if (static_cast<unsigned long long>(p.sides) * p.parts >= (1ull << 32)) return FA_ERR_UNSUPPORTED;
  const unsigned long long warps = static_cast<unsigned long long>(n) * p.sides * p.parts;
  const unsigned long long blocks = (warps + kCopyThreads / 32 - 1) / (kCopyThreads / 32), most = 8ull * sms;
  return static_cast<fa_status>(launch_dependent(pages_copy_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                                                 dim3(kCopyThreads), 0, static_cast<cudaStream_t>(stream), p));
}

fa_status fa_pages_free(const int* block_table, const int* seqlens, const int* rows, const int* shares,
                        int* shares_out, int* freed, int* num_freed, int B, int n, int max_pages, int page_size,
                        int num_pages, void* stream) {
  if (B < 1 || n < 1 || max_pages < 1 || num_pages < 1 || (!rows && n != B)) return FA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(seqlens),
                        static_cast<const void*>(shares), static_cast<const void*>(shares_out),
                        static_cast<const void*>(freed), static_cast<const void*>(num_freed)})
    if (!x || pg_off(x, 4)) return FA_ERR_INVALID_ARG;
  if (pg_off(rows, 4)) return FA_ERR_INVALID_ARG;
  if (page_size != kPgTokens) return FA_ERR_UNSUPPORTED;
  const long long mp = max_pages;
  if (mp * kPgTokens >= (1ll << 31) || mp * B >= (1ll << 31) || mp * n >= (1ll << 31) || num_pages > FA_PAGES_MAX)
    return FA_ERR_UNSUPPORTED;
  SetParams p = {};
  p.cap = mp * n < num_pages ? mp * n : num_pages;
  const PgRange in = {shares, 4ll * num_pages};
  if (pg_meet({{shares_out, 4ll * num_pages}, {freed, 4 * p.cap}, {num_freed, 4}},
              {{block_table, 4 * mp * B}, {seqlens, 4ll * B}, {rows, 4ll * n}, {shares_out == shares ? nullptr : in.p, in.bytes}}))
    return FA_ERR_INVALID_ARG;
  p.table = block_table;
  p.seqlens = seqlens;
  p.rows = rows;
  p.shares = shares;
  p.shares_out = shares_out;
  p.list0 = freed;
  p.counts = num_freed;
  p.B = B;
  p.n = n;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.err = device_error_word();
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (mp * n < kFreeLarge) return static_cast<fa_status>(launch_set<0>(p, cs));
  const int sms = device_sm_count();
  if (!sms) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  auto blocks = [&](long long work) {
    const long long b = (work + kFreeThreads - 1) / kFreeThreads;
    return dim3(static_cast<unsigned>(b < 8ll * sms ? b : 8ll * sms));
  };
  int rc = launch_dependent(pages_free_begin_kernel, blocks(p.cap > num_pages ? p.cap : num_pages), dim3(kFreeThreads), 0, cs, p);
  const long long chunks = (mp + 31) / 32 * n;
  if (rc == FA_OK) rc = launch_dependent(pages_free_count_kernel, blocks((chunks + kSetRows - 1) / kSetRows * 32), dim3(kFreeThreads), 0, cs, p);
  if (rc == FA_OK) rc = launch_set<2>(p, cs);
  return static_cast<fa_status>(rc);
}

fa_status fa_pages_compact(const int* block_table, const int* seqlens, const int* shares, int* table_out,
                           int* shares_out, int* copy_src, int* copy_dst, int* counts, int B, int max_pages,
                           int page_size, int num_pages, int first, void* stream) {
  if (B < 1 || max_pages < 1 || num_pages < 1 || first < 0 || first >= num_pages) return FA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(seqlens),
                        static_cast<const void*>(shares), static_cast<const void*>(table_out),
                        static_cast<const void*>(shares_out), static_cast<const void*>(counts)})
    if (!x || pg_off(x, 4)) return FA_ERR_INVALID_ARG;
  if (page_size != kPgTokens) return FA_ERR_UNSUPPORTED;
  const long long mp = max_pages;
  if (mp * kPgTokens >= (1ll << 31) || mp * B >= (1ll << 31) || num_pages > FA_PAGES_MAX) return FA_ERR_UNSUPPORTED;
  SetParams p = {};
  p.cap = mp * B < (num_pages - first) / 2 ? mp * B : (num_pages - first) / 2;
  if (p.cap > 0 && (!copy_src || !copy_dst)) return FA_ERR_INVALID_ARG;
  if (pg_off(copy_src, 4) || pg_off(copy_dst, 4)) return FA_ERR_INVALID_ARG;
  const long long table = 4 * mp * B, pool = 4ll * num_pages;
  if (pg_meet({{table_out, table}, {shares_out, pool}, {copy_src, 4 * p.cap}, {copy_dst, 4 * p.cap}, {counts, 8}},
              {{seqlens, 4ll * B}, {table_out == block_table ? nullptr : block_table, table},
               {shares_out == shares ? nullptr : shares, pool}}))
    return FA_ERR_INVALID_ARG;
  p.table = block_table;
  p.seqlens = seqlens;
  p.shares = shares;
  p.table_out = table_out;
  p.shares_out = shares_out;
  p.list0 = copy_src;
  p.list1 = copy_dst;
  p.counts = counts;
  p.B = B;
  p.n = B;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.first = first;
  p.err = device_error_word();
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  return static_cast<fa_status>(launch_set<1>(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
