// tree.cu -- attention of a tree of drafted tokens over the paged cache.
//
// What it computes. Sequence b has S = seqlens[b] keys, the last n of which are the
// drafted nodes. Query row i < n is node i: it sees key j if j < S - n (the committed
// text) or bit j - (S - n) of its mask row is set. O = softmax(scale * q K^T) V over
// the keys it sees, lse = ln sum exp; a row that sees none, and rows from n on, get
// O = 0 and lse = -inf; a row with a score of NaN or +inf (a query that is not finite) gets NaN
// for both. A KV head's g = Hq / Hkv query heads times T nodes are R = g * T
// rows, dense in q, o and lse: row r is node r % T of head r / T.
//
// What bounds it. K and V are read once for R rows: R FLOP per byte. Up to some 256
// rows that is HBM time, beyond it the tensor cores'. So the tensor cores run
// (tcgen05, 128 rows a tile) whatever R is: a tile of 128 keys costs a tile of rows
// about 1.1 us of S = Q K^T, softmax and O += P V in a row, and at full HBM rate an SM
// gets such a K/V tile (64 KB at d = 128) every 1.5 us.
//
// How.
//   * Work is cut into equal shares of key tiles, not of sequences: every group of CTAs of
//     the one-per-SM grid sums the batch's cost for itself and takes the share
//     [c N / G, (c+1) N / G) of it. Lengths live on the device and may differ by any
//     factor; every share costs the same within a step. A share that does not
//     cover its (sequence, KV head) whole leaves fp32 partials (O, max, sums) in the
//     workspace, at most two per CTA, and the merge kernel joins them. A list of the
//     split ones, one entry per CTA, tells it which; what is whole is written at once.
//   * The CTAs of a group go over the same keys side by side: KV heads whose rows lie beside
//     one another in a page, and the row units of a head, which share its keys in L2.
//   * R <= 128 (NARROW): two key tiles at a time for the one tile of rows. Softmax
//     warps 0-3 take the even tiles, 4-7 the odd ones, each with its own S/P and O in
//     TMEM, so that one's softmax runs under the other's MMAs; the two are joined in
//     TMEM at the end of a share (a warp can read the other's lanes).
//   * R > 128 (WIDE): two tiles of rows against each key tile, as the prefill kernel.
//   * Small problems (tr_cluster): a unit to a cluster, whose CTAs join their partials
//     through shared memory (one launch, no workspace). Units are not shared out there, so
//     it is for few steps.
//   * warp 8, in narrow units with warp 10: K and V pages by TMA, 16-token boxes through the
//     block table, into rings of 128-byte-swizzled tiles; the Q tile too (rows are dense: one
//     plain box).
//   * warp 9: TMEM and the MMA chain. S_t(x+1) is issued right behind PV_t(x).
//   * the mask is looked at only in tiles that reach past S - n: a thread's row has
//     its 128 bits of the tile in four registers. Rows of padding warps are skipped.
// P is rounded to bf16 for the tensor cores, as in the prefill and decode kernels (by at most
// 2^-8 of a weight; fp32 P would take twice the MMAs of P V, as two bf16 parts), O is rounded
// to bf16 once at the end, all sums and maxima are fp32: O is off by 0.0023 relative, of which
// its own rounding is 0.0017.
// Every mbarrier wait is bounded; a wait that runs out records FA_ERR_TIMEOUT and the
// CTA unwinds. The softmax warps leave together by a vote at the barrier they share.
#include <atomic>
#include <type_traits>

#include "launch.cuh"

namespace fa {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_tiled();  // defined in api.cu

constexpr int kTrTile = 128;  // rows of a tile, keys of a tile

template <int D, bool WIDE>
struct TrCfg {
  static constexpr int KCH = D / 64;             // 64-element (128-byte) chunks along d
  static constexpr int CHUNK_BYTES = 128 * 128;  // 128 rows x 128 bytes, swizzled
  static constexpr int Q_BYTES = kTrTile * D * 2;
  static constexpr int KV_BYTES = kTrTile * D * 2;
  static constexpr int QT = WIDE ? 2 : 1;
  // stages of K and of V: 64 to 96 KB of each in flight (3 + 3 tiles of 32 KB fill the
  // SM's shared memory beside one Q tile; HBM needs about 70 KB in flight an SM)
  static constexpr int STAGES = D == 64 ? (WIDE ? 5 : 6) : (WIDE ? 2 : 3);
  static constexpr int OFF_K = QT * Q_BYTES;
  static constexpr int OFF_V = OFF_K + STAGES * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + STAGES * KV_BYTES;
  static constexpr int OFF_EX = OFF_BAR + 384;
  static constexpr int SMEM = OFF_EX + kTrTile * 5 * 4;  // at most 227 KB; the base is 1024-byte aligned
  // clustered: partials of all rows over Q and the rings, 16 bytes of padding a row against
  // bank conflicts, then their maxima and sums (behind Q, which may still be on its way
  // where a share is empty)
  static constexpr int PART_PITCH = D * 4 + 16;
  static constexpr int OFF_ML = QT * kTrTile * PART_PITCH;
  static_assert(OFF_ML >= OFF_K && OFF_ML + QT * kTrTile * 16 <= OFF_BAR, "partials");
  static constexpr int LEAST = WIDE ? 4 : 1;  // steps of a share
  static constexpr int STEP = WIDE ? 2 : 3, FRONT = WIDE ? 6 : 4;  // TrCost
  static_assert(STEP + FRONT <= 8, "a batch's cost (tr_most_steps)");
  static constexpr int TMEM_COLS = 512;
  static constexpr int SLOT_COLS = 256;  // a slot's columns: S/P, then O
  static constexpr int O_OFF = 128;
  static constexpr int THREADS = 384;  // 2 x 4 softmax warps, producer, MMA issuer, V producer (narrow), an idle warp
  static constexpr int SOFTMAX_REGS = 192;  // 256 * 192 + 128 * 120 = 384 * 168
  static constexpr int AUX_REGS = 120;
  static_assert(SMEM <= 232448, "shared memory of an SM");
};

struct TrParams {
  __nv_bfloat16* o;
  float* lse;  // may be null
  const int* block_table;
  const int* seqlens;
  const int* tree_lens;  // may be null: T nodes each
  const int* mask;
  long long mask_sb;  // words from a sequence's mask to the next's; 0: one for all
  int B, Hkv, T, R, U;  // U: row units of a (sequence, KV head)
  int V, Hv;            // CTAs of a group, which go over the same keys side by side: the row units of
                        // Hv KV heads (V = U * Hv), or 1
  int units;            // of a sequence, for each CTA of a group
  int words;            // of a mask row
  int C;                // CTAs of a cluster (the clustered form)
  int max_pages, num_pages;
  float c;  // scale * log2(e)
  float* part;     // [2 * grid][128 * QT][D]: unnormalised O of partial shares
  float4* part_ml; // [2 * grid][128 * QT]: (max in log2 units, sum as P V saw it, sum, -)
  int4* split;     // [grid]: (first row, rows, partials, -) of the unit that CTA c begins and does not end; z == 0: none
  unsigned* err;
  unsigned long long timeout_ns;
};

// What shares are cut in: `step` for a step and, ahead of a unit's first, `front` for what
// a unit costs beside its tiles (Q, the first S, writing O): 4/3 of a pair of tiles in
// narrow units, 3 tiles in wide ones (64 sequences of up to 2100 keys, d = 128: 92 us with
// starts uncounted, 63 us; 16 of up to 16384, 512 rows, d = 64: 174 us at 1.5 tiles, 166 us
// at 3). Batches of so few steps that a CTA has hardly more than one are cut by steps alone.
struct TrCost {
  int step, front;
  // the steps whose cost ends within the first `at` of a unit
  __device__ __forceinline__ int steps_in(int at) const { return at < front ? 0 : (at - front) / step; }
};

struct TrBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], v_full[6], k_empty[6], v_empty[6];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int finished;  // the clustered form: this CTA's partial is there
  // where this CTA's share begins
  int b0, off0, begin, end, total, grid;
  TrCost cost;
};
static_assert(sizeof(TrBars) <= 384, "barrier area");

// Lengths of a sequence, clamped to what the table and the step hold.
struct TrSeq {
  int S, n;
  int tiles;  // key tiles to go through
};
__device__ __forceinline__ TrSeq tr_seq(const TrParams& p, int b) {
  TrSeq s;
  s.S = max(0, min(__ldg(p.seqlens + b), p.max_pages * 16));
  s.n = max(0, min(p.tree_lens ? __ldg(p.tree_lens + b) : p.T, min(p.T, s.S)));
  s.tiles = s.n > 0 ? (s.S + kTrTile - 1) / kTrTile : 0;
  return s;
}
// Steps of one (KV head, row unit): a key tile, or (narrow) a pair of them; a unit
// without keys is one step, so that somebody writes its zeros.
template <bool WIDE>
__device__ __forceinline__ int tr_steps(const TrSeq& s) {
  return max(1, WIDE ? s.tiles : (s.tiles + 1) / 2);
}

// A run of steps of one unit inside a CTA's share.
struct TrSeg {
  int b, kvh, u;
  int S, n;
  int x0, nt;    // first key tile and how many
  bool from_start, to_end;
  int unit_end;  // where the unit ends in the whole batch's cost
};

// The clustered form: a unit to a cluster, an even run of its steps to each CTA.
template <bool WIDE>
struct TrOne {
  bool done = false;
  __device__ __forceinline__ TrOne(const TrBars*) {}
  __device__ __forceinline__ bool next(const TrParams& p, TrSeg& g) {
    if (done) return false;
    done = true;
    constexpr int PER = WIDE ? 1 : 2;
    const int unit = static_cast<int>(blockIdx.x) / p.C, rank = static_cast<int>(blockIdx.x) - unit * p.C;
    const int bh = unit / p.U;
    g.b = bh / p.Hkv;
    g.kvh = bh - g.b * p.Hkv;
    g.u = unit - bh * p.U;
    const TrSeq q = tr_seq(p, g.b);
    g.S = q.S;
    g.n = q.n;
    const int steps = tr_steps<WIDE>(q), per = (steps + p.C - 1) / p.C;
    g.x0 = min(steps, rank * per) * PER;
    g.nt = max(0, min(q.tiles, min(steps, (rank + 1) * per) * PER) - g.x0);
    g.from_start = g.to_end = p.C == 1;
    g.unit_end = 0;
    return true;
  }
};

// Walks a share segment by segment; each role walks by itself.
template <bool WIDE>
struct TrWalk {
  int b, off, at;  // sequence, cost into it; cost into the batch
  const volatile TrBars* s;  // the rest is read again each time: few registers over the tile loops
  __device__ __forceinline__ TrWalk(const TrBars* bars) : b(bars->b0), off(bars->off0), at(bars->begin), s(bars) {}
  __device__ __forceinline__ bool next(const TrParams& p, TrSeg& g) {
    TrSeq q;
    int cost, hu, from, to, j0, j1;
    const TrCost c = {s->cost.step, s->cost.front};
    const int end = s->end;
    do {
      if (at >= end) return false;
      q = tr_seq(p, b);
      cost = c.front + c.step * tr_steps<WIDE>(q);
      hu = off / cost;
      from = off - hu * cost;
      to = min(cost, from + end - at);
      j0 = c.steps_in(from);
      j1 = c.steps_in(to);
      // a share that ends inside a unit's first step leaves all of it to the next CTA
      if (j0 == j1) at += to - from;
    } while (j0 == j1);
    constexpr int PER = WIDE ? 1 : 2;
    g.b = b;
    if (p.V > 1) {  // the CTA's head (of Hv) and row unit are its place in its group
      const int place = static_cast<int>(blockIdx.x) % p.V;
      g.kvh = hu * p.Hv + place / p.U;
      g.u = place % p.U;
    } else {
      g.kvh = hu / p.U;
      g.u = hu - g.kvh * p.U;
    }
    g.S = q.S;
    g.n = q.n;
    g.x0 = j0 * PER;
    g.nt = max(0, min(q.tiles, j1 * PER) - g.x0);
    g.from_start = j0 == 0;
    g.to_end = to == cost;
    g.unit_end = at - from + cost;
    off += to - from;
    at += to - from;
    if (off == cost * p.units) {
      ++b;
      off = 0;
    }
    return true;
  }
};

// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// 32 bytes in one store: a warp whose threads each write a row of their own spends a
// wavefront per row and store, so half as many as with 16 bytes.
__device__ __forceinline__ void st32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The other CTAs of the cluster: a barrier for all their threads, and reads of their shared
// memory at the place that `p` has in this CTA's.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t in_cta(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ int ld_cluster_int(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ bool vote_all(int id, int nthreads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// 32 visibility bits of a row for keys off .. off + 31, counted from the first node
// (negative: committed text). `row`: the row's mask words, n nodes.
__device__ __forceinline__ uint32_t tr_bits(const int* row, int words, int n, int off) {
  if (off <= -32) return 0xffffffffu;
  if (off >= n) return 0u;
  auto word = [&](int w) -> uint32_t {  // words past the last node are not read
    return w >= 0 && w < words ? static_cast<uint32_t>(__ldg(row + w)) : 0u;
  };
  uint32_t v;
  if (off < 0) {
    v = ((1u << -off) - 1u) | (word(0) << -off);
  } else {
    v = __funnelshift_r(word(off >> 5), word((off >> 5) + 1), off & 31);
  }
  const int left = n - off;  // nodes from here on
  return left < 32 ? v & ((1u << left) - 1u) : v;
}

// A row's partials joined: maximum, sums, and a lane's four columns of O. A partial whose
// maximum is +inf (its scores were NaN) makes all of them NaN.
struct TrRow {
  float m = -INFINITY, s = 0.f, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);  // a lane's four columns
  __device__ __forceinline__ void add(float m2, float s2, float l2, const float4& o2) {
    if (m2 == -INFINITY) return;  // a share without a key that this row sees: its O was not written
    const float mn = fmaxf(m, m2);
    const float fa = ex2_approx(m - mn), fb = ex2_approx(m2 - mn);
    s = s * fa + s2 * fb;
    l = l * fa + l2 * fb;
    o = make_float4(o.x * fa + o2.x * fb, o.y * fa + o2.y * fb, o.z * fa + o2.z * fb, o.w * fa + o2.w * fb);
    m = mn;
  }
};

template <int D, bool WIDE, bool CL>
__global__ void __launch_bounds__(384, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const TrParams p) {
  using C = TrCfg<D, WIDE>;
  using Walk = typename std::conditional<CL, TrOne<WIDE>, TrWalk<WIDE>>::type;
  constexpr int ST = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  TrBars* bars = reinterpret_cast<TrBars*>(smem + C::OFF_BAR);
  float* ex = reinterpret_cast<float*>(smem + C::OFF_EX);  // [5][128]: max and sum of both slots, lse sum of slot 1

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (smem_u32(smem) & 1023u) {  // the swizzle atoms' alignment; the block's only shared memory starts at a multiple
    pdl_wait();
    if (threadIdx.x == 0) {
      record_error(p.err, FA_ERR_TIMEOUT, SITE_TR_SMEM);
      if (!CL) p.split[cta] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 128);
      mbar_init(&bars->pv_done[t], 1);
    }
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    bars->finished = 0;
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(&bars->tmem_base, C::TMEM_COLS);
  pdl_wait();

  // ---- this CTA's share of the batch's cost: a block-wide scan over the sequences
  if constexpr (!CL) {
    const int per = (p.B + C::THREADS - 1) / C::THREADS;
    const int lo = min(p.B, static_cast<int>(threadIdx.x) * per), hi = min(p.B, lo + per);
    int mine = 0;  // a batch's whole cost is below 2^31
    for (int b = lo; b < hi; ++b) mine += tr_steps<WIDE>(tr_seq(p, b));
    const int units = p.units;
    mine *= units;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    // totals per warp go through the exchange area, which nothing uses yet
    int* wsum = reinterpret_cast<int*>(ex);
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = inc - mine, steps = 0;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      if (w < warp) before += wsum[w];
      steps += wsum[w];
    }
    // Each CTA that shares a unit writes, and the merge reads, a partial of its rows, which
    // for 256 rows costs as much as some tiles: a CTA gets LEAST steps at least, but no two
    // units while others get none. A share is a step's cost or more either way, so that every
    // CTA between a unit's first and last has a step of it.
    const int grid = static_cast<int>(gridDim.x) / p.V, me = cta / p.V;  // groups, and this CTA's
    const bool few = steps <= 2 * C::LEAST * grid;
    const TrCost cost = few ? TrCost{1, 0} : TrCost{C::STEP, C::FRONT};
    const int G = few ? min(grid, max(steps / C::LEAST, p.B * units)) : grid;
    const int total = cost.step * steps + cost.front * p.B * units;
    const int begin = me < G ? static_cast<int>(static_cast<long long>(me) * total / G) : total;
    const int end = me < G ? static_cast<int>((me + 1ll) * total / G) : total;
    if (threadIdx.x == 0) {
      bars->begin = begin;
      bars->end = end;
      bars->total = total;
      bars->grid = G;
      bars->cost = cost;
    }
    before = cost.step * before + cost.front * lo * units;
    mine = cost.step * mine + cost.front * (hi - lo) * units;
    if (begin >= before && begin < before + mine) {  // one thread: its sequences hold the share's start
      int off = begin - before;
      int b = lo;
      for (; b < hi; ++b) {
        const int s = (cost.step * tr_steps<WIDE>(tr_seq(p, b)) + cost.front) * units;
        if (off < s) break;
        off -= s;
      }
      bars->b0 = b;
      bars->off0 = off;
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;
  const uint64_t tmo = p.timeout_ns;
  const uint64_t tmo_unwind = unwind_timeout(tmo);
  auto fail = [&](unsigned site) {
    record_error(p.err, FA_ERR_TIMEOUT, site);
    *abort_flag = 1;
  };

  if (warp >= 8) {
    warpgroup_reg_dealloc<C::AUX_REGS>();
    if (warp == 8 || (!WIDE && warp == 10)) {
      // ======================= producers: K (and Q), V =======================
      // Narrow: a warp each. A tile is 8 or 16 boxes of 16 rows per operand, and one warp
      // issuing both spent 650 cycles a tile and 57 a box on it, more than the tile's HBM time
      // at d = 64 (b19 hkv8 s16384 125 -> 107 us; d = 128 the same). Wide: one warp for both,
      // there is time, and a second one's waits take issue slots from two softmax warps (b19
      // hq64 t64 d64 319 us, 339 us with two).
      const bool is_k = warp == 8;
      const CUtensorMap* my_map = is_k ? &tmK : &tmV;
      uint8_t* my_ring = is_k ? sK : sV;
      uint64_t* my_full = is_k ? bars->k_full : bars->v_full;
      uint64_t* my_empty = is_k ? bars->k_empty : bars->v_empty;
      if (lane == 0) {
        if (is_k) tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(my_map);
        if (WIDE) tma_prefetch_desc(&tmV);
      }
      Walk walk(bars);
      TrSeg w;
      uint32_t g = 0;  // key tiles loaded so far (ring position)
      uint32_t q_loads = 0;
      const int pi = lane / C::KCH, pc = lane % C::KCH;  // the box of this lane: page and d-chunk
      bool ok = true;
      while (ok && !*abort_flag && walk.next(p, w)) {
        const int* trow = p.block_table + static_cast<size_t>(w.b) * p.max_pages;
        const int n_pages = (w.S + 15) >> 4;
        // a lane holds one of 32 entries, four tiles' worth; the next 32 are fetched meanwhile
        // (one tile ahead would leave an L2 round trip in every tile)
        auto fetch = [&](int x) -> int {
          const int pg = (w.x0 + x) * 8 + lane;
          return pg < n_pages && pg < (w.x0 + w.nt) * 8 ? __ldg(trow + pg) : -1;
        };
        int ent = -1, ent_next = fetch(0);
        // The last segment's Q is in use until its last S: this one's first tiles go ahead
        // of its Q (all but one stage of the ring, which that segment's own end frees).
        bool q_due = is_k;
        auto load_q = [&]() {
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars->q_full, C::QT * C::Q_BYTES);
            for (int t = 0; t < C::QT; ++t)
              for (int c = 0; c < C::KCH; ++c)
                tma_load_3d(sQ + t * C::Q_BYTES + c * C::CHUNK_BYTES, &tmQ, &bars->q_full, c * 64,
                            (w.u * C::QT + t) * kTrTile, w.b * p.Hkv + w.kvh);
          }
          ++q_loads;
          q_due = false;
        };
        auto q_free = [&]() {  // uniform: every lane asks, and one answer counts
          return q_loads == 0 || __all_sync(0xffffffffu, mbar_test(&bars->q_empty, (q_loads - 1) & 1));
        };
        for (int x = 0; x < w.nt; ++x, ++g) {
          if (q_due) {
            if (q_free()) {
              load_q();
            } else if (x == ST - 1) {
              if (!mbar_wait(&bars->q_empty, (q_loads - 1) & 1, tmo, abort_flag)) {
                ok = false;
                break;
              }
              load_q();
            }
          }
          const int s = g % ST;
          if ((x & 3) == 0) {
            ent = ent_next;
            ent_next = fetch(x + 4);
          }
          const int npg = min(8, n_pages - (w.x0 + x) * 8);  // pages past the end are not loaded
          int pe = __shfl_sync(0xffffffffu, ent, (x & 3) * 8 + (pi & 7));
          if (pi < npg && (pe < 0 || pe >= p.num_pages)) {
            // never dereferenced: page 0 is loaded in its place, the output is undefined
            record_error(p.err, FA_ERR_BOUNDS, SITE_TR_TABLE);
            pe = 0;
          }
          const uint32_t bytes = static_cast<uint32_t>(npg) * 16 * 128 * C::KCH;
          auto load = [&](const CUtensorMap* map, uint8_t* ring, uint64_t* full, uint64_t* empty) -> bool {
            if (g >= ST && !mbar_wait(&empty[s], (g / ST - 1) & 1, tmo, abort_flag)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes);
            __syncwarp();
            if (pi < npg)
              tma_load_3d(ring + s * C::KV_BYTES + pc * C::CHUNK_BYTES + pi * 2048, map, &full[s], pc * 64, w.kvh,
                          pe * 16);
            return true;
          };
          if constexpr (WIDE) {
            ok = load(&tmK, sK, bars->k_full, bars->k_empty);
            if (ok && !load(&tmV, sV, bars->v_full, bars->v_empty)) {
              ok = false;
              mbar_wait(&bars->k_full[s], (g / ST) & 1, tmo_unwind);  // K was issued: let it land
            }
          } else {
            ok = load(my_map, my_ring, my_full, my_empty);
          }
          if (!ok) break;
        }
        if (ok && q_due) {
          if (q_loads > 0 && !mbar_wait(&bars->q_empty, (q_loads - 1) & 1, tmo, abort_flag))
            ok = false;
          else
            load_q();
        }
      }
      if (!ok) fail(SITE_TR_PRODUCER);
      // Copies in flight must land before the CTA exits. Waited for whether or not a wait has
      // run out so far: another role's may after this warp has issued its last copy.
      if (q_loads > 0) mbar_wait(&bars->q_full, (q_loads - 1) & 1, tmo_unwind);
      for (uint32_t x = g > ST ? g - ST : 0; x < g; ++x) {
        mbar_wait(&my_full[x % ST], (x / ST) & 1, tmo_unwind);
        if (WIDE) mbar_wait(&bars->v_full[x % ST], (x / ST) & 1, tmo_unwind);
      }
    } else if (warp == 9) {
      // ======================= MMA issuer =======================
      const bool leader = elect_one();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kTrTile, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem_u32(sV), C::CHUNK_BYTES, 1024);
      // S of slot t = Q (row tile t, or the only one) K^T, K in ring stage st
      auto qk = [=](int t, int st) {
        const uint64_t a0 = dQ + static_cast<uint64_t>((WIDE ? t * C::Q_BYTES : 0) >> 4);
        const uint64_t b0 = dK + static_cast<uint64_t>((st * C::KV_BYTES) >> 4);
        const uint32_t dS = tmem + t * C::SLOT_COLS;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * C::CHUNK_BYTES + (kk & 3) * 32) >> 4);
            tc_mma_ss(dS, a0 + off, b0 + off, idesc_qk, kk > 0 ? 1u : 0u);
          }
        }
      };
      auto pv = [=](int t, int st, bool first) {
        const uint64_t b0 = dV + static_cast<uint64_t>((st * C::KV_BYTES) >> 4);
        const uint32_t dO = tmem + t * C::SLOT_COLS + C::O_OFF;
        const uint32_t aP = tmem + t * C::SLOT_COLS;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kTrTile / 16; ++kk)
            tc_mma_ts(dO, aP + kk * 8, b0 + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv,
                      (!first || kk > 0) ? 1u : 0u);
        }
      };
      auto commit = [=](uint64_t* bar) {
        if (leader) tc_commit(bar);
      };
      auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool { return mbar_wait(bar, parity, tmo, abort_flag); };
      auto wait_k = [&](uint32_t x) -> bool {
        const bool r = wwait(&bars->k_full[x % ST], (x / ST) & 1);
        tc_fence_after();
        return r;
      };
      auto wait_v = [&](uint32_t x) -> bool {
        const bool r = wwait(&bars->v_full[x % ST], (x / ST) & 1);
        tc_fence_after();
        return r;
      };
      uint32_t pph[2] = {0, 0};  // p_full phase parities
      auto wait_p = [&](int t) -> bool {
        const bool r = wwait(&bars->p_full[t], t ? pph[1] : pph[0]);
        if (t) pph[1] ^= 1; else pph[0] ^= 1;
        tc_fence_after();
        return r;
      };
      Walk walk(bars);
      TrSeg w;
      uint32_t g = 0;      // key tiles of earlier segments (ring position)
      uint32_t seg_i = 0;
      bool ok = true;
      for (; ok && walk.next(p, w); ++seg_i, g += w.nt) {
        const int nt = w.nt;
        if (!wwait(&bars->q_full, seg_i & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (nt == 0) {
          if (leader) mbar_arrive(&bars->q_empty);
          continue;
        }
        if constexpr (!WIDE) {
          // slots take the tiles in turn: tile x in slot x & 1
          for (int x = 0; x < 2 && x < nt; ++x) {
            if (!wait_k(g + x)) {
              ok = false;
              break;
            }
            qk(x, (g + x) % ST);
            commit(&bars->s_full[x]);
            commit(&bars->k_empty[(g + x) % ST]);
            if (x + 1 == nt) commit(&bars->q_empty);
          }
          for (int x = 0; ok && x < nt; ++x) {
            const int t = x & 1;
            if (!wait_p(t) || !wait_v(g + x)) {
              ok = false;
              break;
            }
            pv(t, (g + x) % ST, x < 2);
            commit(&bars->v_empty[(g + x) % ST]);
            if (x + 2 >= nt) {
              commit(&bars->pv_done[t]);
            } else {
              // S of this slot overwrites the columns P was read from; one thread's MMAs run in order
              if (!wait_k(g + x + 2)) {
                ok = false;
                break;
              }
              qk(t, (g + x + 2) % ST);
              commit(&bars->s_full[t]);
              commit(&bars->k_empty[(g + x + 2) % ST]);
              if (x + 3 == nt) commit(&bars->q_empty);  // the segment's last S
            }
          }
        } else {
          const bool two = (w.u * 2 + 1) * kTrTile < p.R;  // the unit's second row tile exists
          if (!wait_k(g)) {
            ok = false;
            break;
          }
          qk(0, g % ST);
          commit(&bars->s_full[0]);
          if (two) {
            qk(1, g % ST);
            commit(&bars->s_full[1]);
          }
          commit(&bars->k_empty[g % ST]);
          if (nt == 1) commit(&bars->q_empty);
          for (int x = 0; ok && x < nt; ++x) {
            const int sv = (g + x) % ST, sk = (g + x + 1) % ST;
            const bool more = x + 1 < nt;
            if (!wait_p(0) || !wait_v(g + x)) {
              ok = false;
              break;
            }
            pv(0, sv, x == 0);
            if (!two) commit(&bars->v_empty[sv]);
            if (more) {
              if (!wait_k(g + x + 1)) {
                ok = false;
                break;
              }
              qk(0, sk);
              commit(&bars->s_full[0]);
            } else {
              commit(&bars->pv_done[0]);
            }
            if (two) {
              if (!wait_p(1)) {
                ok = false;
                break;
              }
              pv(1, sv, x == 0);
              commit(&bars->v_empty[sv]);
              if (more) {
                qk(1, sk);
                commit(&bars->s_full[1]);
              } else {
                commit(&bars->pv_done[1]);
              }
            }
            if (more) {
              commit(&bars->k_empty[sk]);
              if (x + 2 == nt) commit(&bars->q_empty);
            }
          }
        }
      }
      if (!ok && leader) fail(SITE_TR_MMA);
      commit(&bars->drain);  // every MMA must finish before TMEM is released
      mbar_wait(&bars->drain, 0, tmo_unwind);
    }
    if (CL && p.C > 1) {  // the partials are there; they have been read
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ======================= softmax: warps 0-3 (slot 0), 4-7 (slot 1) =======================
    warpgroup_reg_alloc<C::SOFTMAX_REGS>();
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;  // row of the tile == TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + t * C::SLOT_COLS;
    const uint32_t tO = tS + C::O_OFF;
    const float2 c2 = make_float2(p.c, p.c);
    // The reference maximum m is raised only when a row's maximum climbs more than this
    // above it; until then the exponentials stay below 2^8 and carry one constant factor
    // that O / l cancels.
    constexpr float kRescaleSlack = 8.f;
    bool ok = true;
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, tmo, abort_flag));
    };
    Walk walk(bars);
    TrSeg w;
    uint32_t cnt = 0;   // tiles of this slot done so far (s_full phases)
    uint32_t ecnt = 0;  // segments with at least one tile in this slot (pv_done phases)
    uint32_t gkv = 0;   // ring position at the segment's start
    bool listed = false;
    while (walk.next(p, w)) {
      const int row = WIDE ? (w.u * 2 + t) * kTrTile + r : r;  // of the R rows
      const bool has_rows = row - lane < p.R;                  // some row of this warp exists (warp-uniform)
      const bool tile_exists = !WIDE || (w.u * 2 + t) * kTrTile < p.R;
      // The row's node, -1 if it has none. Formed anew where it is needed, in masked tiles and
      // at the segment's end: kept over the loop below, it and the mask's address are spilled.
      auto node_of = [&]() {
        int x = row;
        asm volatile("" : "+r"(x));
        const int node = x % p.T;
        return x < p.R && node < w.n ? node : -1;
      };
      const int base = w.S - w.n;  // first node's key
      const int step = WIDE ? 1 : 2;
      const int x_first = WIDE ? 0 : t;
      const int mine = !tile_exists || w.nt <= x_first ? 0 : (w.nt - x_first + step - 1) / step;  // tiles of this slot
      float m = -INFINITY;
      float l = 0.f;   // sum of the unrounded p: the lse's
      float lc = 0.f;  // bf16(p_top) - p_top of each tile's largest p, rescaled like l

      for (int i = 0; i < mine; ++i, ++cnt) {
        const int x = x_first + i * step;  // tile of the segment
        const int key0 = (w.x0 + x) * kTrTile;
        const bool masked = key0 + kTrTile > base;
        uint32_t bits[4];  // fetched while S is being computed
        if (masked) {
          const int node = node_of();
          const int* mrow = p.mask + w.b * p.mask_sb + static_cast<size_t>(max(node, 0)) * p.words;
#pragma unroll
          for (int wd = 0; wd < 4; ++wd) bits[wd] = node >= 0 ? tr_bits(mrow, p.words, w.n, key0 + 32 * wd - base) : 0u;
        }
        if (!wwait(&bars->s_full[t], cnt & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (has_rows) {
          uint32_t raw[4][32];
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS + cc * 32, raw[cc]);
          tmem_ld_wait();
          float s[128];
#pragma unroll
          for (int k = 0; k < 128; ++k) s[k] = __uint_as_float(raw[k >> 5][k & 31]);
          if (masked) {
#pragma unroll
            for (int k = 0; k < 128; ++k)
              if (!((bits[k / 32] >> (k % 32)) & 1u)) s[k] = -INFINITY;
          }
          float mx8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float a = fmax3(s[16 * k], s[16 * k + 1], s[16 * k + 2]);
#pragma unroll
            for (int e = 3; e < 15; e += 2) a = fmax3(a, s[16 * k + e], s[16 * k + e + 1]);
            mx8[k] = fmaxf(a, s[16 * k + 15]);
          }
          const float mx = fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
          const float m_tile = mx * p.c;
          const float m_new = (m_tile > m + kRescaleSlack) ? m_tile : m;
          const float m_use = (m_new == -INFINITY) ? 0.f : m_new;
          const float alpha = ex2_approx(m - m_use);
          // the largest p is not 1 against a stale reference: O's normaliser counts it as
          // the bf16 product sees it, so that a nearly one-hot row is not off by its rounding
          const float p_top = ex2_approx(fmaf(mx, p.c, -m_use));
          const float p_top_err = __bfloat162float(__float2bfloat16_rn(p_top)) - p_top;
          const float2 nm2 = make_float2(-m_use, -m_use);
          float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int e = cc * 32 + 2 * k;
              const float2 v = ffma2(make_float2(s[e], s[e + 1]), c2, nm2);
              const float2 ev = make_float2(ex2_approx(v.x), ex2_approx(v.y));
              acc[k & 3] = fadd2(acc[k & 3], ev);
              pk[k] = pack_bf16x2(ev.x, ev.y);
            }
            tmem_st16(tS + cc * 16, pk);
          }
          const float2 at = fadd2(fadd2(acc[0], acc[1]), fadd2(acc[2], acc[3]));
          l = fmaf(l, alpha, at.x + at.y);
          lc = fmaf(lc, alpha, p_top_err);
          m = m_new;
          // PV of this slot's previous tile is complete: S of this one was issued behind it
          if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            const float2 al2 = make_float2(alpha, alpha);
#pragma unroll
            for (int cc = 0; cc < D / 32; cc += 2) {
              uint32_t o0[32], o1[32];
              tmem_ld32(tO + cc * 32, o0);
              tmem_ld32(tO + cc * 32 + 32, o1);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 v0 = fmul2(make_float2(__uint_as_float(o0[k]), __uint_as_float(o0[k + 1])), al2);
                const float2 v1 = fmul2(make_float2(__uint_as_float(o1[k]), __uint_as_float(o1[k + 1])), al2);
                o0[k] = __float_as_uint(v0.x);
                o0[k + 1] = __float_as_uint(v0.y);
                o1[k] = __float_as_uint(v1.x);
                o1[k + 1] = __float_as_uint(v1.y);
              }
              tmem_st32(tO + cc * 32, o0);
              tmem_st32(tO + cc * 32 + 32, o1);
            }
          }
        }
        // V rows past the sequence's end hold whatever the pool or an earlier tile left
        // there, and 0 * NaN is not 0: the slot whose PV on this tile comes first zeroes them
        if (key0 + kTrTile > w.S && (!WIDE || t == 0)) {
          const uint32_t xg = gkv + x;
          if (!wwait(&bars->v_full[xg % ST], (xg / ST) & 1)) {
            ok = false;
            break;
          }
          uint8_t* vt = sV + (xg % ST) * C::KV_BYTES;
          const int r0 = w.S - key0;
          for (int idx = r; idx < (kTrTile - r0) * C::KCH * 8; idx += 128) {
            const int vr = r0 + idx / (C::KCH * 8);
            const int rem = idx % (C::KCH * 8);
            *reinterpret_cast<uint4*>(vt + (rem >> 3) * C::CHUNK_BYTES + vr * 128 + (rem & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->p_full[t]);
      }
      gkv += w.nt;
      if (ok && mine > 0) {
        if (!wwait(&bars->pv_done[t], ecnt & 1)) ok = false;
        ++ecnt;
        tc_fence_after();
      }
      if (!ok) fail(SITE_TR_SOFTMAX);

      // ---- the segment's end: final rows, or a partial
      const bool live = node_of() >= 0;
      if (!live) {
        m = -INFINITY;
        l = lc = 0.f;
      }
      // A score that is NaN (a query that is not finite) may have left m at -inf, which would
      // weigh the row 0: at +inf its weight, 2^(m - m), is NaN, here and in every join.
      if (l != l) m = INFINITY;
      const bool whole = w.from_start && w.to_end;
      const int slot = 2 * cta + (w.from_start ? 1 : 0);
      const size_t out_row = (static_cast<size_t>(w.b) * p.Hkv + w.kvh) * p.R + row;
      const size_t part_row = static_cast<size_t>(slot) * (kTrTile * C::QT) + (WIDE ? t * kTrTile : 0) + r;
      if (!CL && threadIdx.x == 0 && w.from_start && !w.to_end && ok) {
        // this CTA begins the unit: the last group with a share of it is the one whose share holds its end
        const long long last = (static_cast<long long>(w.unit_end) * bars->grid - 1) / bars->total;
        const int first_row = w.u * C::QT * kTrTile;
        p.split[cta] = make_int4((w.b * p.Hkv + w.kvh) * p.R + first_row, min(p.R - first_row, C::QT * kTrTile),
                                 static_cast<int>(last) - cta / p.V + 1, 0);
        listed = true;
      }
      float m_all = m, sum = l + lc, lsum = l;
      float f0 = 1.f, f1 = 0.f;  // weights of this slot's O (wide), or of slot 0's and slot 1's (narrow)
      if constexpr (!WIDE) {
        ex[t * 128 + r] = m;
        ex[(2 + t) * 128 + r] = l + lc;
        if (t == 1) ex[4 * 128 + r] = l;
        ok = vote_all(1, 256, ok);
        if (!ok) break;  // all eight warps leave in the same segment
        const float m0 = ex[r], m1 = ex[128 + r];
        m_all = fmaxf(m0, m1);
        const float m_use = m_all == -INFINITY ? 0.f : m_all;
        f0 = ex2_approx(m0 - m_use);
        f1 = ex2_approx(m1 - m_use);
        sum = f0 * ex[256 + r] + f1 * ex[384 + r];
        if (t == 0) lsum = f0 * l + f1 * ex[512 + r];
      } else if (CL) {
        // (a partial goes where the other slot's MMAs read their operands)
        ok = vote_all(1, 256, ok);
        if (!ok) break;
      } else if (!ok) {
        break;
      }
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (NaN stays NaN)
        f0 *= inv;
        f1 *= inv;
      }
      if (has_rows && tile_exists) {
        // narrow: each slot's warps write half the columns of the joined O
        constexpr int COLS = WIDE ? D : D / 2;
        const int col0 = WIDE ? 0 : t * COLS;
        const bool take0 = (WIDE ? mine > 0 : w.nt > 0) && f0 != 0.f;
        const bool take1 = !WIDE && w.nt > 1 && f1 != 0.f;
        const uint32_t o_base = tmem + lane_base + (WIDE ? t * C::SLOT_COLS : 0) + C::O_OFF;
        const bool write = row < p.R;
#pragma unroll
        for (int cc = 0; cc < COLS / 32; ++cc) {
          uint32_t a[32], b[32];
          tmem_ld32(o_base + col0 + cc * 32, a);
          if constexpr (!WIDE) tmem_ld32(o_base + C::SLOT_COLS + col0 + cc * 32, b);
          tmem_ld_wait();
          float o[32];
          // TMEM that no PV wrote, and rows whose weight is 0 over whatever P held, are not taken in
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            o[k] = take0 ? f0 * __uint_as_float(a[k]) : 0.f;
            if constexpr (!WIDE) o[k] = take1 ? fmaf(f1, __uint_as_float(b[k]), o[k]) : o[k];
          }
          if (!write) continue;
          if (whole) {
            // (o may start on any 16-byte border)
            __nv_bfloat16* dst = p.o + out_row * D + col0 + cc * 32;
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<uint4*>(dst + 8 * q) =
                  live ? make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                                    pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]))
                       : make_uint4(0u, 0u, 0u, 0u);
          } else if (CL) {
            if (m_all != -INFINITY) {  // else its weight is 0 and nobody reads it (nor has Q necessarily come)
              float* dst = reinterpret_cast<float*>(smem + (WIDE ? t * kTrTile + r : r) * C::PART_PITCH) + col0 + cc * 32;
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4*>(dst + 4 * q) = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          } else if (live) {
            float* dst = p.part + part_row * D + col0 + cc * 32;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(o[8 * q + k]);
              st32(dst + 8 * q, v);
            }
          }
        }
        if (write && (WIDE || t == 0)) {
          if (whole) {
            if (p.lse) p.lse[out_row] = lsum == 0.f ? -INFINITY : (m_all + log2f(lsum)) * kLn2;
          } else {
            float4* ml = CL ? reinterpret_cast<float4*>(smem + C::OFF_ML) + (WIDE ? t * kTrTile + r : r) : p.part_ml + part_row;
            *ml = make_float4(m_all, sum, lsum, 0.f);
          }
        }
      }
      tc_fence_before();
      // narrow: both slots' O have been read by all before either is overwritten, and the
      // exchange area before the next segment fills it
      if constexpr (!WIDE) named_bar_sync(2, 256);
    }
    if (!CL && threadIdx.x == 0 && !listed) p.split[cta] = make_int4(0, 0, 0, 0);
    if (CL && p.C > 1) {
      // Joined inside the cluster: each CTA reads its part of the rows out of all CTAs' shared
      // memory. (These warps: the others have given their registers away.)
      if (threadIdx.x == 0) bars->finished = ok;  // as all eight warps voted
      cluster_sync();
      constexpr int LANES = D / 4, PER = 32 / LANES;  // lanes to a row, rows of a warp's load
      const int rank = cta % p.C;
      const int unit_rows = min(p.R - w.u * C::QT * kTrTile, C::QT * kTrTile);
      const int per = (unit_rows + p.C - 1) / p.C, last = min(unit_rows, (rank + 1) * per);
      const int my = lane / LANES, col = lane % LANES * 4;
      bool all = true;
      for (int c = 0; c < p.C; ++c) all &= ld_cluster_int(in_cta(&bars->finished, c)) != 0;
      for (int row = rank * per + warp * PER + my; all && row < last; row += 8 * PER) {
        TrRow acc;
        for (int c0 = 0; c0 < p.C; c0 += 4) {  // four CTAs' loads in flight
          float4 ml[4], o[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c0 + c >= p.C) continue;
            ml[c] = ld_cluster(in_cta(smem + C::OFF_ML + row * 16, c0 + c));
            o[c] = ld_cluster(in_cta(smem + row * C::PART_PITCH + col * 4, c0 + c));
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c0 + c < p.C) acc.add(ml[c].x, ml[c].y, ml[c].z, o[c]);
        }
        const float inv = acc.s == 0.f ? 0.f : 1.f / acc.s;
        const size_t out = (static_cast<size_t>(w.b) * p.Hkv + w.kvh) * p.R + w.u * C::QT * kTrTile + row;
        *reinterpret_cast<uint2*>(p.o + out * D + col) =
            make_uint2(pack_bf16x2(acc.o.x * inv, acc.o.y * inv), pack_bf16x2(acc.o.z * inv, acc.o.w * inv));
        if (p.lse && col == 0) p.lse[out] = acc.l == 0.f ? -INFINITY : (acc.m + log2f(acc.l)) * kLn2;
      }
      cluster_sync();  // nobody leaves while others read its shared memory
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Joins the partials of the units that several CTAs share: lse = log2 sum 2^(m_s - m) l_s
// + m, O = sum 2^(m_s - m) O_s / sum 2^(m_s - m) l_s. Every block makes the list of split
// units from the CTAs' entries (in their order, so that all agree), keeps it in shared
// memory and takes items of it in turn. What a row costs is round trips to L2, so: units
// of two partials go two rows to a lane group, all of them in flight; the others one row
// to 1, 2, 4 or 8 warps (as many as the rows leave warps for), four partials of each in
// flight.
constexpr int kTrMaxGrid = 1024;  // CTAs the list has room for
constexpr int kTrFewParts = 2;
constexpr int kTrMergeBlocks = 3;  // per SM

struct TrUnit {
  int first_item, row0, rows, parts;
};

// Block-wide inclusive scan of 256 values; *total gets their sum.
__device__ __forceinline__ int scan256(int v, int* warp_sum, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, k);
    if (lane >= k) v += y;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k < warp) v += warp_sum[k];
    all += warp_sum[k];
  }
  __syncthreads();
  *total = all;
  return v;
}

template <int D, int QT>
__global__ void __launch_bounds__(256, kTrMergeBlocks) tree_merge_kernel(const float* __restrict__ part,
                                                                         const float4* __restrict__ part_ml,
                                                                         const int4* __restrict__ split, int grid,
                                                                         int V,
                                                                         __nv_bfloat16* __restrict__ o,
                                                                         float* __restrict__ lse) {
  constexpr int LANES = D / 4;           // lanes to a row
  constexpr int PER = 32 / LANES;        // rows of a warp's load
  constexpr int ROWS = kTrTile * QT;
  __shared__ TrUnit unit[kTrMaxGrid];  // by CTA; those of CTAs without an entry have no items
  __shared__ int warp_sum[8];
  __shared__ float4 red[8][32];
  __shared__ float red_m[8][PER], red_s[8][PER], red_l[8][PER];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  int many_rows = 0;  // rows of units with more than a few partials
  for (int c0 = 0; c0 < grid; c0 += 256) {
    const int c = c0 + threadIdx.x;
    TrUnit u = {0, 0, 0, 0};
    if (c < grid) {
      const int4 un = split[c];
      u = {0, un.x, un.z > 0 ? un.y : 0, un.z};
      unit[c] = u;
    }
    int sum;
    scan256(u.parts > kTrFewParts ? u.rows : 0, warp_sum, &sum);
    many_rows += sum;
  }
  int wpr = 8;  // warps to a row
  while (wpr > 1 && many_rows / PER * wpr > 8 * static_cast<int>(gridDim.x)) wpr >>= 1;
  const int few_rows = 8 * 2 * PER, many_step = 8 / wpr * PER;  // rows of an item
  const int my = lane / LANES, col = lane % LANES * 4;
  int total = 0;
  for (int c0 = 0; c0 < grid; c0 += 256) {
    const int c = c0 + threadIdx.x;
    int items = 0;
    if (c < grid) {
      const int per = unit[c].parts > kTrFewParts ? many_step : few_rows;
      items = (unit[c].rows + per - 1) / per;
    }
    int sum;
    const int inc = scan256(items, warp_sum, &sum);
    if (c < grid) unit[c].first_item = total + inc - items;
    total += sum;
  }
  __syncthreads();
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    int c = 0, hi = grid;  // the last entry that begins at or before the item: entries without items begin with the next
    while (hi - c > 1) {
      const int mid = (c + hi) / 2;
      if (unit[mid].first_item <= item) c = mid; else hi = mid;
    }
    const TrUnit un = unit[c];
    // partial 0 is CTA c's last, the others are the first of the later groups' CTAs
    auto at = [&](int i) { return static_cast<size_t>(i == 0 ? 2 * c + 1 : 2 * (c + i * V)) * ROWS; };
    auto get = [&](float4& ml, float4& v, size_t row_at) {
      ml = part_ml[row_at];
      v = *reinterpret_cast<const float4*>(part + row_at * D + col);
    };
    auto put = [&](const TrRow& r, int row) {
      const float inv = r.s == 0.f ? 0.f : 1.f / r.s;
      const size_t out = static_cast<size_t>(un.row0) + row;
      *reinterpret_cast<uint2*>(o + out * D + col) =
          make_uint2(pack_bf16x2(r.o.x * inv, r.o.y * inv), pack_bf16x2(r.o.z * inv, r.o.w * inv));
      if (lse && col == 0) lse[out] = r.l == 0.f ? -INFINITY : (r.m + log2f(r.l)) * kLn2;
    };
    if (un.parts <= kTrFewParts) {
      const int row0 = (item - un.first_item) * few_rows + warp * 2 * PER + my;
      TrRow acc[2];
      float4 ml[kTrFewParts][2], v[kTrFewParts][2];
#pragma unroll
      for (int k = 0; k < kTrFewParts; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          ml[k][r] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
          if (k < un.parts && row0 + r * PER < un.rows) get(ml[k][r], v[k][r], at(k) + row0 + r * PER);
        }
#pragma unroll
      for (int k = 0; k < kTrFewParts; ++k)
#pragma unroll
        for (int r = 0; r < 2; ++r) acc[r].add(ml[k][r].x, ml[k][r].y, ml[k][r].z, v[k][r]);
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (row0 + r * PER < un.rows) put(acc[r], row0 + r * PER);
    } else {
      constexpr int IN = 4;
      const int sub = warp & (wpr - 1);
      const int row = (item - un.first_item) * many_step + warp / wpr * PER + my;
      TrRow acc;
      for (int i0 = sub; i0 < un.parts; i0 += wpr * IN) {
        float4 ml[IN], v[IN];
#pragma unroll
        for (int k = 0; k < IN; ++k) {
          ml[k] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
          if (i0 + wpr * k < un.parts && row < un.rows) get(ml[k], v[k], at(i0 + wpr * k) + row);
        }
#pragma unroll
        for (int k = 0; k < IN; ++k) acc.add(ml[k].x, ml[k].y, ml[k].z, v[k]);
      }
      if (wpr > 1) {  // block-uniform
        red[warp][lane] = acc.o;
        if (col == 0) {
          red_m[warp][my] = acc.m;
          red_s[warp][my] = acc.s;
          red_l[warp][my] = acc.l;
        }
        __syncthreads();
        if (sub == 0)
          for (int k = warp + 1; k < warp + wpr; ++k) acc.add(red_m[k][my], red_s[k][my], red_l[k][my], red[k][lane]);
        __syncthreads();
      }
      if (sub == 0 && row < un.rows) put(acc, row);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
static bool tr_wide(int R) { return R > kTrTile; }

// The most steps that a batch can have, 0 where their cost could reach 2^31.
static long long tr_most_steps(int B, int Hkv, int R, int max_pages) {
  const long long U = tr_wide(R) ? (R + 2ll * kTrTile - 1) / (2 * kTrTile) : 1;
  const long long tiles = (static_cast<long long>(max_pages) * 16 + kTrTile - 1) / kTrTile;
  const long long steps = tr_wide(R) ? tiles : (tiles + 1) / 2;
  const long long n = static_cast<long long>(B) * Hkv * U;
  return n > (1ll << 31) / 8 / steps ? 0 : n * steps;  // STEP + FRONT <= 8
}

// CTAs of a launch: one to an SM, none that could have no step.
static int tr_grid(long long steps, int sms) { return static_cast<int>(steps < sms ? steps : sms); }

// The clustered form for small problems: a unit to a cluster of C CTAs, which join their
// partials through shared memory. It saves the share scan, the second launch and the
// partials' way through L2 (b1 hkv8 t8 d128, s1000 8.4 us against 11.3, s8000 12.8 against
// 15.0; b4 s2000 10.8 against 16.4), but takes no more than C of the SMs for a unit and
// counts with the longest context the table allows: taken where that leaves a CTA about as
// many steps as equal shares over all SMs would. One sequence, whose units are all of one
// length, may take a few more (t8 hkv8 s24000, 8 steps for 5: d128 22.0 against 22.4 us, d64
// 16.2 against 18.0; hkv4 s16000, 6 for 2: 18.3 against 15.9 us).
//   In a batch one sequence may fill its row of the table and the others be short; their SMs
// are idle while its clusters go through it, so a CTA gets few steps there. At the most that
// the rule takes, one long sequence among short ones costs up to a quarter more than equal
// shares, and a batch of long ones a tenth to a third less (d128, us, clusters / shares, one
// long and all long: narrow b19 hkv8 s2048, 8 steps, 17.6 / 15.9 and 28.9 / 32.6; b19 hkv4
// s2560, 5 steps, 14.9 / 12.3 and 17.0 / 21.4; wide b19 hkv8 s1280, 10 steps, 21.1 / 21.3 and
// 27.3 / 31.3; b19 hkv4 s2048, 8 steps, 25.9 / 20.7 and 27.6 / 34.1; b4 hkv8 s4096, 8 steps,
// 23.1 / 29.6 and 23.9 / 35.8). Past it: narrow b19 hkv8 s8192 57.7 / 20.9 and 95.9 / 99.5.
// Returns C, 0 for the general form.
constexpr int kTrMaxCluster = 12;
static int tr_cluster(long long steps, int B, int Hkv, int R, int sms) {
  // clusters of 1, 2, .. 12 of these CTAs that run at once on 152 SMs, by the driver's
  // occupancy query on one GPU: a cluster needs SMs of one GPC, and its GPCs had 16 to 20.
  // Where another GPU's are cut otherwise, clusters too many wait for a second wave.
  static const int fit[kTrMaxCluster] = {152, 76, 46, 36, 28, 23, 15, 15, 15, 13, 8, 8};
  const bool wide = tr_wide(R);
  const long long U = wide ? (R + 2ll * kTrTile - 1) / (2 * kTrTile) : 1;
  const long long units = static_cast<long long>(B) * Hkv * U, of_unit = steps / units;
  int most = 0;
  while (most < kTrMaxCluster && units * 152 <= static_cast<long long>(fit[most]) * sms) ++most;
  if (most == 0) return 0;
  const long long per = (of_unit + most - 1) / most, shared = (steps + sms - 1) / sms;
  const int C = static_cast<int>((of_unit + per - 1) / per);  // no more CTAs than the steps need
  long long most_steps = shared + (wide ? 3 : B == 1 ? 2 : 1);
  if (B == 1 && shared >= 4) ++most_steps;
  const long long ragged = C == 1 ? (wide ? 10 : 8) : (wide ? 8 : 5);
  if (B > 1 && most_steps > ragged) most_steps = ragged;
  return per <= most_steps ? C : 0;
}

static size_t tr_part_bytes(int grid, int R, int d) {
  return static_cast<size_t>(2) * grid * (tr_wide(R) ? 256 : 128) * d * 4;
}
static size_t tr_ml_bytes(int grid, int R) { return static_cast<size_t>(2) * grid * (tr_wide(R) ? 256 : 128) * 16; }

template <int D, bool WIDE, bool CL>
static int launch_tree(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const TrParams& p,
                       int grid, cudaStream_t stream) {
  using C = TrCfg<D, WIDE>;
  auto kfn = tree_kernel<D, WIDE, CL>;
  // the attributes hold for the life of the device's context: asked for once per device
  static std::atomic<unsigned long long> asked{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda_failure(e);
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e == cudaSuccess && CL) e = cudaFuncSetAttribute(kfn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return record_cuda_failure(e);
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  if (CL) return launch_dependent_cluster(kfn, dim3(grid), p.C, dim3(C::THREADS), C::SMEM, stream, tq, tk, tv, p);
  int rc = launch_dependent(kfn, dim3(grid), dim3(C::THREADS), C::SMEM, stream, tq, tk, tv, p);
  if (rc != FA_OK) return rc;
  const int merge_grid = kTrMergeBlocks * grid;
  return launch_dependent(tree_merge_kernel<D, C::QT>, dim3(merge_grid), dim3(256), 0, stream,
                          static_cast<const float*>(p.part), static_cast<const float4*>(p.part_ml),
                          static_cast<const int4*>(p.split), grid, p.V, p.o, p.lse);
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_tree_workspace_bytes(int B, int Hq, int Hkv, int T, int max_pages, int d, int num_sms) {
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || max_pages < 1 || d < 1 || num_sms < 1 || Hq % Hkv != 0) return 0;
  const long long R = static_cast<long long>(Hq / Hkv) * T;
  if (R >= (1ll << 31)) return 0;
  const long long steps = tr_most_steps(B, Hkv, static_cast<int>(R), max_pages);
  if (steps == 0) return 0;
  if (tr_cluster(steps, B, Hkv, static_cast<int>(R), num_sms)) return 0;
  const int grid = tr_grid(steps, num_sms);
  return tr_part_bytes(grid, static_cast<int>(R), d) + tr_ml_bytes(grid, static_cast<int>(R)) +
         static_cast<size_t>(grid) * 16;
}

fa_status fa_tree_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                               const int* seqlens, const int* tree_mask, int mask_shared, const int* tree_lens,
                               void* o, float* lse, int B, int Hq, int Hkv, int T, int max_pages, int page_size,
                               int num_pages, int d, float scale, void* workspace, size_t ws_bytes, void* stream) {
  auto mis = [](const void* x, uintptr_t m) { return (reinterpret_cast<uintptr_t>(x) & (m - 1)) != 0; };
  if (!q || !k_pages || !v_pages || !block_table || !seqlens || !tree_mask || !o) return FA_ERR_INVALID_ARG;
  if (mis(q, 16) || mis(k_pages, 16) || mis(v_pages, 16) || mis(o, 16) || mis(block_table, 4) || mis(seqlens, 4) ||
      mis(tree_mask, 4) || (tree_lens && mis(tree_lens, 4)) || (lse && mis(lse, 4)) || mis(workspace, 256))
    return FA_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || max_pages < 1 || num_pages < 1 || Hq % Hkv != 0 || !(scale > 0.f) ||
      !(scale < INFINITY))
    return FA_ERR_INVALID_ARG;
  if (page_size != 16 || (d != 64 && d != 128)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * 16 >= (1ll << 31) ||
      static_cast<long long>(max_pages) * 16 > (1ll << 31) - 256 || static_cast<long long>(B) * Hq * T >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;  // (a key's index, rounded up to whole tiles, is a 32-bit number)
  {
    // o, lse and the workspace are written while other CTAs still read the rest
    const long long rows = static_cast<long long>(B) * Hq * T, q_bytes = rows * d * 2;
    const long long pool = 32ll * num_pages * Hkv * d, b4 = 4ll * B;
    const struct { const void* p; long long n; } out[] = {{o, q_bytes}, {lse, rows * 4}, {workspace, static_cast<long long>(ws_bytes)}},
        in[] = {{q, q_bytes}, {k_pages, pool}, {v_pages, pool}, {block_table, b4 * max_pages}, {seqlens, b4},
                {tree_lens, b4}, {tree_mask, 4ll * (mask_shared ? 1 : B) * T * ((T + 31ll) / 32)}};
    for (int i = 0; i < 3; ++i) {
      for (const auto& x : in)
        if (overlap(out[i].p, out[i].n, x.p, x.n)) return FA_ERR_INVALID_ARG;
      for (int k = 0; k < i; ++k)
        if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return FA_ERR_INVALID_ARG;
    }
  }
  const int R = Hq / Hkv * T;
  const long long steps = tr_most_steps(B, Hkv, R, max_pages);
  if (steps == 0) return FA_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  if (!sms) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  if (sms > kTrMaxGrid) return FA_ERR_UNSUPPORTED;
  const size_t need = fa_tree_workspace_bytes(B, Hq, Hkv, T, max_pages, d, sms);
  if (ws_bytes < need || (need && !workspace)) return FA_ERR_INVALID_ARG;
  const int cluster = tr_cluster(steps, B, Hkv, R, sms);
  const int grid = cluster ? B * Hkv * (tr_wide(R) ? (R + 2 * kTrTile - 1) / (2 * kTrTile) : 1) * cluster : tr_grid(steps, sms);
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return FA_ERR_CUDA;

  CUtensorMap tq, tk, tv;
  {
    // a KV head's R rows are dense; rows past R read as zeros
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)R, (cuuint64_t)B * Hkv};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)R * d * 2};
    cuuint32_t box[3] = {64, 128, 1};
    cuuint32_t es[3] = {1, 1, 1};
    if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return static_cast<fa_status>(record_cuda_failure(cudaErrorInvalidValue));
  }
  for (int i = 0; i < 2; ++i) {
    // one 16-token page of one KV head per box; L2 fetches what a row is, no neighbour's
    const CUtensorMapL2promotion fetch = d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hkv, (cuuint64_t)num_pages * 16};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)Hkv * d * 2};
    cuuint32_t box[3] = {64, 1, 16};
    cuuint32_t es[3] = {1, 1, 1};
    if (enc(i == 0 ? &tk : &tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(i == 0 ? k_pages : v_pages),
            dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return static_cast<fa_status>(record_cuda_failure(cudaErrorInvalidValue));
  }
  TrParams p;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.tree_lens = tree_lens;
  p.mask = tree_mask;
  p.words = (T + 31) / 32;
  p.mask_sb = mask_shared ? 0 : static_cast<long long>(T) * p.words;
  p.B = B;
  p.Hkv = Hkv;
  p.T = T;
  p.R = R;
  p.U = tr_wide(R) ? (R + 2 * kTrTile - 1) / (2 * kTrTile) : 1;
  // Side by side: the row units of a KV head, which read the same keys (from L2 all but once:
  // b19 hq64 hkv8 t64 s16384 d128 420 us, 455 us one after the other), and as many KV heads
  // as fit, whose keys lie beside one another in a page (b38 hq64 hkv8 t8 s8192 d64 104 us,
  // 112 us one after the other). Up to 16 CTAs, and groups that leave few SMs over.
  p.V = p.Hv = 1;
  if (p.U <= 8)
    for (int h = Hkv; h >= 1; --h) {
      const int v = h * p.U;
      if (Hkv % h == 0 && v <= 16 && v <= grid && grid % v <= grid / 24) {
        p.V = v;
        p.Hv = h;
        break;
      }
    }
  p.units = p.V > 1 ? Hkv / p.Hv : Hkv * p.U;
  p.C = cluster;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.c = scale * kLog2e;
  p.part = nullptr;
  p.part_ml = nullptr;
  p.split = nullptr;
  if (!cluster) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.part = reinterpret_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float4*>(ws + tr_part_bytes(grid, R, d));
    p.split = reinterpret_cast<int4*>(ws + tr_part_bytes(grid, R, d) + tr_ml_bytes(grid, R));
  }
  p.err = device_error_word();
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  p.timeout_ns = wait_timeout_ns();
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  auto go = [&](auto wide, auto cl) {
    constexpr bool W = decltype(wide)::value, CL = decltype(cl)::value;
    return d == 128 ? launch_tree<128, W, CL>(tq, tk, tv, p, grid, cs) : launch_tree<64, W, CL>(tq, tk, tv, p, grid, cs);
  };
  const std::true_type yes{};
  const std::false_type no{};
  const int rc = tr_wide(R) ? (cluster ? go(yes, yes) : go(yes, no)) : (cluster ? go(no, yes) : go(no, no));
  return static_cast<fa_status>(rc);
}

}  // extern "C"
