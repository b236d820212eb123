// paged_plan.cu -- what a step over the paged cache needs before its first kernel:
// block tables, slot maps and positions from request lengths, and the visibility
// mask and positions of a tree of drafted tokens from its parent indexes.
//
// fa_paged_plan. Sequence b holds c = cached[b] tokens and gets n = new_lens[b] more.
// It holds have = ceil(c / 16) pages and needs want = ceil((c + n) / 16). The pages
// come from the front of the free list, sequence by sequence:
//   block_table[b][have + i] = free_pages[first_b + i],  i < want - have,
//   first_b = sum over b' < b of (want_b' - have_b').
// The new token at position p = c + t goes to slot block_table[b][p / 16] * 16 + p % 16.
//
// How: one launch without any exchange between blocks. A block owns SEQS sequences
// (one warp each) and sums the needs of every sequence before them by itself: 2 * B
// lengths from L2, which for some thousand sequences costs less than a second launch
// or a chain of flags between blocks. The slot of a token on a new page is formed from
// the free list and not from the table entry that some warp is writing at that moment,
// so blocks that share a sequence (blockIdx.y cuts long chunks) need no order. Bound by
// launch latency for decode steps, by the 8 bytes written per token for prefill steps.
//
// fa_tree_mask. sees(i) = {i} + sees(parent(i)). Trees of up to 128 nodes: a thread per
// node, and every round joins to its set that of the node its own ends at, so that the
// rounds are the logarithm of the depth and not the depth. Larger ones (their sets do not
// fit in registers): a thread walks up the parents in shared memory; as parent(i) < i the
// visited bits fall, so it keeps one 32-bit word and stores it (and the empty ones it
// skips) when the walk leaves it. Bound by the deepest walk, 0.15 us an ancestor (a chain of
// 1024 nodes 156 us, of 8192 1.25 ms), or by its stores, a row apart from lane to lane (random
// trees of 8192 nodes: one 34 us, sixteen 186 us, 0.72 TB/s).
#include <initializer_list>

#include "launch.cuh"

namespace fa {

constexpr int kPage = 16;
constexpr int kMostPages = (1 << 27) - 1;  // a pool's: its slots are 32-bit numbers
constexpr int kPlanSeqs = 8;          // sequences per block, one warp each
constexpr int kPlanThreads = kPlanSeqs * 32;
constexpr int kPlanRows = 4;          // tokens of a lane, their loads in flight together
constexpr int kPlanChunk = kPlanRows * 32;  // tokens of a sequence per block
static_assert(FA_PLAN_MAX_T == 65535 * kPlanChunk, "blockIdx.y counts a sequence's chunks");

struct PlanParams {
  const int* cached;
  const int* new_lens;
  const int* free_pages;
  int* block_table;
  int* seqlens;
  int* slots;
  int* positions;
  int* pages_used;
  int B, T, max_pages, num_free, align_end;
  unsigned* err;
};

// A sequence's lengths, clamped to what its table row and the T rows of a step hold.
struct PlanSeq {
  int c, n;
  bool clamped;
};
__device__ __forceinline__ PlanSeq plan_seq(const PlanParams& p, int b) {
  const int cap = p.max_pages * kPage;
  const int c0 = __ldg(p.cached + b), n0 = __ldg(p.new_lens + b);
  PlanSeq s;
  s.c = max(0, min(c0, cap));
  s.n = max(0, min(n0, min(p.T, cap - s.c)));
  s.clamped = s.c != c0 || s.n != n0;
  return s;
}
__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPage - 1) / kPage; }

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanParams p) {
  __shared__ int partial[kPlanSeqs];
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b0 = blockIdx.x * kPlanSeqs;
  const int b = b0 + warp;
  // needs of every sequence before this block's, then of the block's own before this warp's
  int sum = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < b0; i += kPlanThreads) {
    const PlanSeq s = plan_seq(p, i);
    sum += pages_of(s.c + s.n) - pages_of(s.c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) partial[warp] = sum;
  __syncthreads();
  int before = lane < kPlanSeqs ? partial[lane] : 0;
  if (lane < warp && b0 + lane < p.B) {
    const PlanSeq s = plan_seq(p, b0 + lane);
    before += pages_of(s.c + s.n) - pages_of(s.c);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  if (b >= p.B) return;
  const PlanSeq s = plan_seq(p, b);
  const int have = pages_of(s.c), want = pages_of(s.c + s.n);
  int* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
  if (blockIdx.y == 0) {
    bool short_of = s.clamped;
    for (int i = lane; i < want - have; i += 32) {
      const int at = before + i;
      const bool ok = at < p.num_free;
      short_of |= !ok;
      row[have + i] = ok ? __ldg(p.free_pages + at) : -1;
    }
    if (short_of) record_error(p.err, FA_ERR_BOUNDS, SITE_PLAN);
    if (lane == 0) {
      p.seqlens[b] = s.c + s.n;
      if (b == p.B - 1) *p.pages_used = before + want - have;
    }
  }
  // rows of the step: token t sits in row t, or (align_end) in row T - n + t
  const int lead = p.align_end ? p.T - s.n : 0;
  const int r0 = blockIdx.y * kPlanChunk + lane;
  const size_t out = static_cast<size_t>(b) * p.T;
  int page[kPlanRows];
#pragma unroll
  for (int i = 0; i < kPlanRows; ++i) {
    const int t = r0 + 32 * i - lead;
    page[i] = -1;
    if (t >= 0 && t < s.n) {
      const int pg = (s.c + t) / kPage;
      const int at = before + pg - have;
      if (pg < have)
        page[i] = row[pg];  // an entry that no block of this launch writes
      else if (at < p.num_free)
        page[i] = __ldg(p.free_pages + at);
    }
  }
#pragma unroll
  for (int i = 0; i < kPlanRows; ++i) {
    const int r = r0 + 32 * i, t = r - lead;
    if (r >= p.T) continue;
    const bool live = t >= 0 && t < s.n;
    p.slots[out + r] = page[i] >= 0 && page[i] < kMostPages ? page[i] * kPage + (s.c + t) % kPage : -1;
    p.positions[out + r] = live ? s.c + t : 0;
  }
}

// What a block knows of its tree, with the lengths clamped as the attention call clamps them.
struct TreeLens {
  int S, n;
};
__device__ __forceinline__ TreeLens tree_lens_of(const int* seqlens, const int* tree_lens, int b, int T) {
  TreeLens l;
  l.S = max(0, __ldg(seqlens + b));
  l.n = max(0, min(tree_lens ? __ldg(tree_lens + b) : T, min(T, l.S)));
  return l;
}
__device__ __forceinline__ int parent_of(const int* prow, int i, unsigned* err) {
  const int q = __ldg(prow + i);
  if (q >= -1 && q < i) return q;
  record_error(err, FA_ERR_BOUNDS, SITE_TREE_MASK);  // not a tree: the node becomes a root
  return -1;
}

template <int W>
__global__ void __launch_bounds__(128) tree_mask_small_kernel(const int* __restrict__ parents,
                                                              const int* __restrict__ seqlens,
                                                              const int* __restrict__ tree_lens,
                                                              int* __restrict__ mask, int* __restrict__ positions,
                                                              int T, unsigned* err) {
  __shared__ unsigned set[W][128];
  __shared__ int up[128];
  pdl_wait();
  pdl_launch();
  const int b = blockIdx.y, i = threadIdx.x;
  const TreeLens l = tree_lens_of(seqlens, tree_lens, b, T);
  // mine: the nodes from i up to, but without, `at`
  int at = i < l.n ? parent_of(parents + static_cast<size_t>(b) * T, i, err) : -1;
  unsigned mine[W];
#pragma unroll
  for (int w = 0; w < W; ++w) mine[w] = i < l.n && i / 32 == w ? 1u << (i & 31) : 0u;
  while (__syncthreads_or(at >= 0)) {
    up[i] = at;
#pragma unroll
    for (int w = 0; w < W; ++w) set[w][i] = mine[w];
    __syncthreads();
    if (at >= 0) {
#pragma unroll
      for (int w = 0; w < W; ++w) mine[w] |= set[w][at];
      at = up[at];
    }
  }
  if (i >= T) return;
  const size_t row = static_cast<size_t>(b) * T + i;
  int seen = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    mask[row * W + w] = static_cast<int>(mine[w]);
    seen += __popc(mine[w]);
  }
  positions[row] = i < l.n ? l.S - l.n + seen - 1 : 0;
}

constexpr int kTreeMaxNodes = FA_TREE_MASK_MAX_T;  // parents of one sequence in shared memory

__global__ void __launch_bounds__(128) tree_mask_kernel(const int* __restrict__ parents,
                                                        const int* __restrict__ seqlens,
                                                        const int* __restrict__ tree_lens, int* __restrict__ mask,
                                                        int* __restrict__ positions, int T, unsigned* err) {
  extern __shared__ int up[];
  pdl_wait();
  pdl_launch();
  const int b = blockIdx.y;
  const int first = blockIdx.x * blockDim.x;
  const int last = min(T, first + static_cast<int>(blockDim.x));  // nodes before it are all a walk from here visits
  const TreeLens l = tree_lens_of(seqlens, tree_lens, b, T);
  const int n = l.n;
  const int* prow = parents + static_cast<size_t>(b) * T;
  for (int i = threadIdx.x; i < min(last, n); i += blockDim.x) up[i] = parent_of(prow, i, err);
  __syncthreads();
  const int i = first + threadIdx.x;
  if (i >= T) return;
  const int words = (T + 31) / 32;
  int* out = mask + (static_cast<size_t>(b) * T + i) * words;
  int at_word = words - 1;
  unsigned cur = 0;
  int depth = -1;
  for (int at = i < n ? i : -1; at >= 0; at = up[at], ++depth) {
    const int w = at >> 5;
    for (; at_word > w; --at_word) {
      out[at_word] = static_cast<int>(cur);
      cur = 0;
    }
    cur |= 1u << (at & 31);
  }
  for (; at_word >= 0; --at_word) {
    out[at_word] = static_cast<int>(cur);
    cur = 0;
  }
  positions[static_cast<size_t>(b) * T + i] = i < n ? l.S - n + depth : 0;
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_paged_plan(const int* cached, const int* new_lens, const int* free_pages, int num_free, int* block_table,
                        int* seqlens, int* slots, int* positions, int* pages_used, int B, int T, int max_pages,
                        int page_size, int align_end, void* stream) {
  auto bad = [](const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3u); };
  if (bad(cached) || bad(new_lens) || bad(block_table) || bad(seqlens) || bad(slots) || bad(positions) ||
      bad(pages_used))
    return FA_ERR_INVALID_ARG;
  if (num_free < 0 || (num_free > 0 && bad(free_pages))) return FA_ERR_INVALID_ARG;
  if (B < 1 || T < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (page_size != kPage) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * T >= (1ll << 31) || static_cast<long long>(B) * max_pages >= (1ll << 31) ||
      static_cast<long long>(max_pages) * kPage >= (1ll << 31) || T > FA_PLAN_MAX_T)
    return FA_ERR_UNSUPPORTED;
  {
    // blocks read the lengths and the free list of all sequences while others write theirs
    const long long b4 = 4ll * B, bt4 = b4 * T;
    const struct { const void* p; long long n; } in[] = {{cached, b4}, {new_lens, b4}, {free_pages, 4ll * num_free}},
        out[] = {{block_table, b4 * max_pages}, {seqlens, b4}, {slots, bt4}, {positions, bt4}, {pages_used, 4}};
    for (int i = 0; i < 5; ++i) {
      for (const auto& x : in)
        if (overlap(out[i].p, out[i].n, x.p, x.n)) return FA_ERR_INVALID_ARG;
      for (int k = 0; k < i; ++k)
        if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return FA_ERR_INVALID_ARG;
    }
  }
  PlanParams p;
  p.cached = cached;
  p.new_lens = new_lens;
  p.free_pages = free_pages;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.slots = slots;
  p.positions = positions;
  p.pages_used = pages_used;
  p.B = B;
  p.T = T;
  p.max_pages = max_pages;
  p.num_free = num_free;
  p.align_end = align_end ? 1 : 0;
  p.err = device_error_word();
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  const dim3 grid((B + kPlanSeqs - 1) / kPlanSeqs, (T + kPlanChunk - 1) / kPlanChunk);
  return static_cast<fa_status>(
      launch_dependent(paged_plan_kernel, grid, dim3(kPlanThreads), 0, static_cast<cudaStream_t>(stream), p));
}

fa_status fa_tree_mask(const int* parents, const int* seqlens, const int* tree_lens, int* mask, int* positions, int B,
                       int T, void* stream) {
  auto bad = [](const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 3u); };
  if (bad(parents) || bad(seqlens) || bad(mask) || bad(positions) || (tree_lens && bad(tree_lens)))
    return FA_ERR_INVALID_ARG;
  if (B < 1 || T < 1) return FA_ERR_INVALID_ARG;
  if (B > FA_TREE_MASK_MAX_B || T > kTreeMaxNodes) return FA_ERR_UNSUPPORTED;
  {
    const long long b4 = 4ll * B, bt4 = b4 * T, m4 = bt4 * ((T + 31) / 32);
    for (const void* x : {static_cast<const void*>(mask), static_cast<const void*>(positions)}) {
      const long long n = x == mask ? m4 : bt4;
      if (overlap(x, n, parents, bt4) || overlap(x, n, seqlens, b4) || overlap(x, n, tree_lens, b4))
        return FA_ERR_INVALID_ARG;
    }
    if (overlap(mask, m4, positions, bt4)) return FA_ERR_INVALID_ARG;
  }
  unsigned* err = device_error_word();
  if (!err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (T <= 128) {
    const int words = (T + 31) / 32;
    auto kfn = words == 1 ? tree_mask_small_kernel<1>
                          : (words == 2 ? tree_mask_small_kernel<2>
                                        : (words == 3 ? tree_mask_small_kernel<3> : tree_mask_small_kernel<4>));
    return static_cast<fa_status>(launch_dependent(kfn, dim3(1, B), dim3(words * 32), 0, cs, parents, seqlens,
                                                   tree_lens, mask, positions, T, err));
  }
  return static_cast<fa_status>(launch_dependent(tree_mask_kernel, dim3((T + 127) / 128, B), dim3(128),
                                                 static_cast<size_t>(T) * sizeof(int), cs, parents, seqlens, tree_lens,
                                                 mask, positions, T, err));
}

}  // extern "C"
