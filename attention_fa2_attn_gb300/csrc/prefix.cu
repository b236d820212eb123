// prefix.cu -- attention of a batch over the paged cache whose sequences share a prefix, with
// the shared keys read once for all of a group.
//
// What it computes. Row i of sequence b sees keys j <= S - T + i (causal; else j < S), S =
// seqlens[b], exactly as fa_decode_paged. A group is a run of sequences whose first P keys lie
// on the same pages. The softmax over [0, S) is joined from one over [0, P), whose keys are
// read through the group's first row of the table for all of its rows at once, and one over
// [P, S), read through the sequence's own row:
//   m = max(m1, m2), l = 2^(m1 - m) l1 + 2^(m2 - m) l2, O = (2^(m1 - m) O1 + 2^(m2 - m) O2) / l.
//
// What bounds it. A KV head's Hq / Hkv heads and T positions of n sequences are n g T rows
// against each shared key: 64 sequences of 8 heads each make 512 FLOP per byte, where one alone
// has 8. So the prefix costs tensor-core and softmax time, what a sequence has of its own HBM
// time.
//
// How. 128 rows a tile on the tensor cores, one CTA to an SM, equal shares of the batch's cost
// whatever the lengths, partials joined by a second kernel.
//   * An item is a group (its prefix) or a sequence (its own keys). Its row tiles hold the
//     rows of as many whole sequences as fit, in q's order, so one 4-D box brings a tile of Q:
//     [sequences][R rows] behind one another. With R > 128 a sequence is several tiles.
//   * Two row tiles make a wide unit, which goes over the keys with one tile of keys against
//     both. A last tile alone, and own keys of more than 16 rows, are narrow units: two tiles of
//     keys at a time, each with its own S, P and O. Own keys of up to 16 rows are slim units, on
//     warp-level MMAs (px_slim).
//   * A share is a stretch of the line of all units' costs, groups first. One warp walks it ahead
//     of the others and leaves its segments in a queue in shared memory. It takes no part in the
//     scan of the costs: meanwhile it runs a step of no consequence, which fetches its code (0.6 us).
//   * The CTAs that are neighbours take the KV heads of one cost line side by side.
//   * A share of a unit leaves fp32 partials at (the rows before the unit + 256 times the
//     CTA's number): no two shares meet there, since along the line either the unit or the CTA
//     goes up. A sequence without a prefix whose keys lie in one share is written at once.
//   * Code and spills cost more than usual: what a CTA runs for the first time comes from L2 while
//     that is busy, and a spilled value waits in a busy L1. So few unrolled
//     copies, one loop to a kind of segment, and no spills at 208 and 88 registers.
// Measured, both kernels in a graph, d = 128 but where it says 64: 8 sequences of 2000 + 1..200
// keys, 32 over 8 heads, 12.6 us (the launches, the lengths' scan and the first keys are 5);
// 64 of 16384 + 9..1024, 64 over 8 heads, 59.4 us, for 205 MB of keys (231 to 255 MB from DRAM: two
// units of 256 rows go over the prefix, on CTAs that are not at the same keys), where the paged
// decode takes 548; 48 in 6 groups of 4000 + 4..1500, T = 4, 64 over 4 heads, d = 64, 34.0 us (63.6);
// 32 of 1000 + up to 8192, 16 heads, 167.6 us, 6.6 TB/s (233). Prompts are bound by the tensor cores
// and their softmax alone, and fa_decode_paged is faster: 8 of 512 positions behind 8192 keys, 64 over
// 8 heads, 920 us (725), at d = 64 730 (600). Prefix steps are bound by a step's S, softmax and PV
// behind one another (1.6 us for 256 rows and 128 keys, two steps under way), own keys by HBM where
// they are long and by the units' ends where they are short.
// Tried and taken back: two slim units at a time, four warps on each (62 and 167 us); a slim unit's
// Q with its first keys, and the next segment's table entries fetched ahead (58.9 and 168.8).
// P is rounded to bf16 for the tensor cores (by at most 2^-8 of a weight; fp32 would take twice
// the MMAs), O once at the end; sums and maxima are fp32.
// Every mbarrier wait is bounded (one for a whole segment by as much for each of its tiles); a
// wait that runs out records FA_ERR_TIMEOUT and the CTA unwinds. A warp's lanes leave together,
// and the softmax warps by a vote in every unit.
#include <atomic>

#include "groups.h"
#include "join.cuh"
#include "launch.cuh"
#include "warp_mma.cuh"

namespace fa {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_tiled();  // defined in api.cu

constexpr int kPxTile = 128;  // rows of a tile, keys of a tile
constexpr int kPxUnit = 2 * kPxTile;  // rows of a unit, at most
constexpr int kPxSlim = 16;           // rows of a sequence whose own keys are taken as slim units, at most

template <int D>
struct PxCfg {
  static constexpr int KCH = D / 64;
  static constexpr int CHUNK_BYTES = 128 * 128;
  static constexpr int Q_BYTES = kPxTile * D * 2;
  static constexpr int KV_BYTES = kPxTile * D * 2;
  // what the SM's shared memory holds beside two Q tiles; K runs ahead of V by a step anyway
  static constexpr int K_STAGES = D == 64 ? 6 : 3, V_STAGES = D == 64 ? 6 : 2;
  static constexpr int OFF_K = 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + K_STAGES * KV_BYTES;
  static constexpr int OFF_BAR = OFF_V + V_STAGES * KV_BYTES;
  static constexpr int OFF_EX = OFF_BAR + 512;
  static constexpr int SMEM = OFF_EX + kPxTile * 5 * 4;
  static_assert(SMEM <= 232448, "shared memory of an SM");
  // sequences whose lengths fit into the rings beside the most groups, before the rings are in use
  static constexpr int MOST_LENS = (OFF_BAR - OFF_K) / 4 - 2 * FA_PREFIX_MAX_GROUPS - 1;
  static_assert(MOST_LENS > 0, "the groups");
  static_assert(8 * 8 * D * 4 <= Q_BYTES, "slim: eight warps' O for eight rows, in the second Q tile");
  static constexpr int SLOT_COLS = 256;  // a slot's columns: S/P, then O
  static constexpr int O_OFF = 128;
  static constexpr int THREADS = 384;  // 2 x 4 softmax warps, K producer, MMA issuer, V producer, the walk
  static constexpr int SOFTMAX_REGS = 208;  // 256 * 208 + 128 * 88 = 384 * 168
  static constexpr int AUX_REGS = 88;
};

// What shares are cut in: `step` for a step of a unit and, ahead of its first, `front` for what
// it costs beside its keys.
struct PxCost {
  int narrow_step, narrow_front, wide_step, wide_front, own_step, own_front;  // own: narrow or slim
};
#define PX_BY_STEPS PxCost{1, 0, 1, 0, 1, 0}
constexpr int kPxMostCost = 28;  // of a step with its unit's start

struct PxParams {
  __nv_bfloat16* o;
  float* lse;  // may be null
  const int* block_table;
  const int* seqlens;
  const int* starts;       // [G + 1]
  const int* prefix_lens;  // [G]
  int B, G, Hkv, T, R, causal;
  int spt;    // sequences of a row tile (1 where R > 128)
  int TS;     // row tiles of a sequence (1 where R <= 128)
  int r_mul, t_mul;  // floor(2^16 / R) + 1, of T: x times that >> 16 is x / R for x < 128 and R <= 128
  int V;      // KV heads side by side
  int units;  // KV heads of each of these places
  int max_pages, num_pages;
  float c;  // scale * log2(e)
  PxCost cost;
  long long area;   // rows of partials of one place and kind
  long long part_rows;  // 2 kinds * V * area
  float* part;      // [D / 8][part_rows][8]: unnormalised O; the rows of a tile lie side by side, so that lanes
                    // with a row each write whole lines (rows of D, 32 bytes a lane: 4.3 us a tile pair; 2 so)
  float4* part_ml;  // (max in log2 units, sum as P V saw it, sum, -)
  int2* desc;       // [2 kinds][B][Hkv][TS]: (first CTA << 16 | CTAs, first row), or kPxDone
  unsigned* err;
  unsigned long long timeout_ns;
};
constexpr int kPxDone = -1;  // the rows are written

// Where share c of `shares` begins on a line of cost `total`: c * total / shares, in 32 bits.
struct PxCut {
  int whole, rest, shares;
  __device__ __forceinline__ PxCut(int total = 0, int n = 1) : whole(total / n), rest(total % n), shares(n) {}
  __device__ __forceinline__ int begin(int c) const { return c * whole + static_cast<int>(static_cast<unsigned>(c * rest) / static_cast<unsigned>(shares)); }
};

// A run of steps of one unit inside a CTA's share, as all roles get it.
struct PxSeg {
  int s0, n;   // the item's sequences
  int k0, k1;  // its keys
  int tile;    // first row tile of the unit
  int hu;      // KV head of the place
  int x0, nt;  // first key tile and how many; none: the share is done
  int flags;
  int ctas;    // CTAs that share the unit, from the one that begins it on (known to that one)
  int kvh, me;    // KV head, this CTA's number on its line
  int out, part;  // of a sequence's own keys: its first row in the output, and (but for 256 * me) of its partials
  __device__ __forceinline__ bool wide() const volatile { return flags & 1; }
  __device__ __forceinline__ bool own() const volatile { return flags & 2; }  // a sequence's own keys
  __device__ __forceinline__ bool from_start() const volatile { return flags & 4; }
  __device__ __forceinline__ bool to_end() const volatile { return flags & 8; }
};
constexpr int kPxQueue = 3;  // segments on their way from the warp that walks the share to the others
constexpr int kPxWalker = 11;   // the warp that walks
constexpr int kPxReaders = 11;  // warps that take them: producers, MMA issuer, softmax

struct PxBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], v_full[6], k_empty[6], v_empty[6];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t drain;
  uint64_t seg_full[kPxQueue], seg_empty[kPxQueue];
  uint32_t tmem_base;
  int abort_flag;
  int it0, off0, group0;  // where this CTA's share begins
  PxSeg seg[kPxQueue];
};
static_assert(sizeof(PxBars) <= 512, "barrier area");

__device__ __forceinline__ int px_len(const PxParams& p, int b) {
  return max(0, min(__ldg(p.seqlens + b), p.max_pages * 16));
}
// Keys that a group reads once: whole pages, of two sequences or more, which its first one has.
__device__ __forceinline__ int px_prefix(const PxParams& p, int s0, int s1, int asked) {
  return group_of_several(s0, s1, p.B) ? max(0, min(asked, px_len(p, s0))) & ~15 : 0;
}

// A group's prefix or a sequence's own keys.
struct PxItem {
  int s0, s1;  // its sequences
  int k0, k1;  // its keys
  int tiles;   // row tiles
  bool own;    // a sequence's own keys
  __device__ __forceinline__ int key_tiles() const { return k1 > k0 ? (k1 - k0 + kPxTile - 1) / kPxTile : 0; }
  // cost of a wide and of a narrow unit, and of a KV head's units together
  __device__ __forceinline__ int wide(const PxCost& c) const { return c.wide_front + c.wide_step * key_tiles(); }
  __device__ __forceinline__ int narrow(const PxCost& c) const {
    const int pairs = (key_tiles() + 1) / 2;
    return own ? c.own_front + c.own_step * pairs : c.narrow_front + c.narrow_step * pairs;
  }
  __device__ __forceinline__ int head(const PxCost& c) const {
    return k1 > k0 ? tiles / 2 * wide(c) + (tiles & 1) * narrow(c) : 0;
  }
};
__device__ __forceinline__ PxItem px_group(const PxParams& p, int s0, int s1, int prefix) {
  const int n = prefix > 0 ? s1 - s0 : 0;  // (a group without one has no units, and its ends may be anything)
  return PxItem{s0, s1, 0, prefix, p.R <= kPxTile ? (n + p.spt - 1) / p.spt : n * p.TS, false};
}
__device__ __forceinline__ PxItem px_sequence(const PxParams& p, int b, int prefix) {
  return PxItem{b, b + 1, prefix, px_len(p, b), p.TS, true};
}

// The group that b is in, the last that begins at or before it: its first and last sequence
// and its prefix for a sequence in it, 0 for others. `g`: a group at or before it.
__device__ __forceinline__ int px_prefix_of(const PxParams& p, int b, int& g) {
  if (g + 1 < p.G && __ldg(p.starts + g + 1) <= b) {
    int step = 1;  // the next one, or one far ahead: in steps twice as long each, then half as long
#pragma unroll 1
    for (; g + step < p.G && __ldg(p.starts + g + step) <= b; step *= 2) g += step;
#pragma unroll 1
    while (step /= 2)
      if (g + step < p.G && __ldg(p.starts + g + step) <= b) g += step;
  }
  const int s0 = __ldg(p.starts + g), s1 = __ldg(p.starts + g + 1);
  return b >= s0 && b < s1 ? px_prefix(p, s0, s1, __ldg(p.prefix_lens + g)) : 0;
}

// Walks a share segment by segment. Items: the groups, then the sequences.
struct PxWalk {
  int it, off, at, g;  // item, cost into it, cost into the line, the group that is looked at
  int end;
  PxCut cut;
  bool no_groups;
  PxCost c;
  const PxItem* first;  // the item that the share begins in; null: it is past that
  __device__ __forceinline__ PxItem item(const PxParams& p, int i) {
    if (i < p.G) {
      const int s0 = __ldg(p.starts + i), s1 = __ldg(p.starts + i + 1);
      return no_groups ? PxItem{0, 0, 0, 0, 0, false} : px_group(p, s0, s1, px_prefix(p, s0, s1, __ldg(p.prefix_lens + i)));
    }
    return px_sequence(p, i - p.G, no_groups ? 0 : px_prefix_of(p, i - p.G, g));
  }
  // The first item from i on that may have a cost; those without lie in runs (groups of one sequence,
  // rows of a padded batch), and one after the other they are 0.2 us each (32 sequences of 500-3000 keys
  // with 512 empty ones in their middle: 137 us, 51 so; 42 without them). A whole warp.
  __device__ __forceinline__ int with_cost(const PxParams& p, int i) const {
    while (true) {
      const int x = i + static_cast<int>(threadIdx.x & 31);
      bool maybe = true;  // (behind the last as well)
      if (x < p.G) {
        maybe = !no_groups && px_prefix(p, __ldg(p.starts + x), __ldg(p.starts + x + 1), __ldg(p.prefix_lens + x)) > 0;
      } else if (x - p.G < p.B) {
        // (of the groups only the one that is looked at is asked)
        const int b = x - p.G, len = px_len(p, b);
        maybe = len > 0;
        if (maybe && !no_groups) {
          const int s0 = __ldg(p.starts + g), s1 = __ldg(p.starts + g + 1);
          maybe = b < s0 || b >= s1 || len > px_prefix(p, s0, s1, __ldg(p.prefix_lens + g));
        }
      }
      const unsigned found = __ballot_sync(0xffffffffu, maybe);
      if (found) return i + __ffs(found) - 1;
      i += 32;
    }
  }
  __device__ __forceinline__ bool next(const PxParams& p, int me, PxSeg& w) {
    PxItem x;
    int from, to, j0, j1, cost, unit_end;
    bool wide;
#pragma unroll 1
    do {
      if (at >= end) return false;
      x = first ? *first : item(p, it);
      first = nullptr;
      const int head = x.head(c);
      if (head == 0) {  // nothing to do (its cost is 0)
        it = with_cost(p, it + 1);
        off = 0;
        j0 = j1 = 0;
        continue;
      }
      // (a division is some 40 instructions in a row: none where the answer is plain)
      w.hu = p.units > 1 ? off / head : 0;
      const int rest = off - w.hu * head, pair = x.wide(c), u = x.tiles < 2 ? 0 : min(x.tiles / 2, rest / pair);
      w.tile = 2 * u;
      wide = u < x.tiles / 2;
      from = rest - u * pair;
      cost = wide ? pair : x.narrow(c);
      to = min(cost, from + end - at);
      const int step = wide ? c.wide_step : x.own ? c.own_step : c.narrow_step;
      const int front = wide ? c.wide_front : x.own ? c.own_front : c.narrow_front;
      j0 = from <= front ? 0 : (from - front) / step;
      j1 = to == cost ? (wide ? x.key_tiles() : (x.key_tiles() + 1) / 2) : to < front ? 0 : (to - front) / step;
      unit_end = at - from + cost;
      w.flags = (wide ? 1 : 0) | (x.own ? 2 : 0) | (j0 == 0 ? 4 : 0) | (to == cost ? 8 : 0);
      off += to - from;
      at += to - from;
      if (off == head * p.units) {
        ++it;
        off = 0;
      }
      // a share that ends inside a unit's first step leaves all of it to the next CTA
    } while (j0 == j1);
    const int per = wide ? 1 : 2;
    w.s0 = x.s0;
    w.n = x.s1 - x.s0;
    w.k0 = x.k0;
    w.k1 = x.k1;
    w.x0 = j0 * per;
    w.nt = min(x.key_tiles(), j1 * per) - w.x0;
    // CTAs up to the one whose share holds the unit's end
    w.ctas = 1;
    if (!(w.flags & 8)) {
#pragma unroll 1
      while (cut.begin(me + w.ctas) < unit_end) ++w.ctas;
    }
    return true;
  }
};

// What bounds a wait for all of a segment: each of its tiles may take as long as any other wait.
__device__ __forceinline__ uint64_t px_bound(uint64_t tmo, int tiles) {
  return tmo >> 38 ? tmo : tmo * static_cast<uint64_t>(tiles + 2);  // (longer ones than four minutes are long enough)
}

// Takes the segments that the walking warp leaves, one after the other. A segment stays where
// it is until `done`, and its parts are read from there when they are needed: in registers they
// are spilled by the loops over the keys, to memory that a busy L1 has no room for.
struct PxTake {
  uint32_t i = 0;
  // a whole warp; null: the wait ran out
  __device__ __forceinline__ const volatile PxSeg* next(PxBars* bars, uint64_t tmo, const volatile int* abort_flag) const {
    const uint32_t e = i % kPxQueue;
    const volatile PxSeg* at = &bars->seg[e];
    // (where it is not there yet, it comes when the last of the readers has done the one in its place)
    const uint32_t parity = (i / kPxQueue) & 1;
    auto there = [&]() -> bool {
      return __all_sync(0xffffffffu, mbar_test(&bars->seg_full[e], parity)) ||
             __all_sync(0xffffffffu, mbar_wait_lean(&bars->seg_full[e], parity, px_bound(tmo, at->nt), abort_flag));
    };
    return there() ? at : nullptr;
  }
  __device__ __forceinline__ void done(PxBars* bars) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->seg_empty[i % kPxQueue]);
    ++i;
  }
};

// A segment of a sequence's own keys for up to 16 rows, by the eight softmax warps alone. What
// decides here is latency: with 128 rows a tile, 8 of them in use, a unit cost 3 us beside its
// keys and a tile 0.75 us, of which the tensor cores had little. So warp-level MMAs, as in the
// decode kernel: a warp takes 16 keys of every tile with a running maximum, sum and O of its
// own, and no warp waits for another until the unit's end, where the eight are joined through
// shared memory, eight rows at a time. The maximum is the keys' own, never a stale one, so that a
// warp's largest weight is 1, which bf16 holds: px_rows' correction of it has nothing to do here.
// Returns what all eight warps voted.
template <int D>
__device__ __forceinline__ bool px_slim(const PxParams& p, const volatile PxSeg* w, PxBars* bars, uint8_t* sQ, uint8_t* sK,
                                        uint8_t* sV, float* ex, uint32_t seg_i, uint32_t& gkv, uint64_t tmo) {
  using C = PxCfg<D>;
  constexpr int KST = C::K_STAGES, VST = C::V_STAGES;
  const volatile int* abort_flag = &bars->abort_flag;
  int tid = threadIdx.x;
  asm volatile("" : "+r"(tid));  // (as in px_rows)
  const int warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;  // row of the MMA fragment (and + 8), column pair
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_lean(bar, parity, tmo, abort_flag));
  };
  // keys that the thread's two rows see (what rows from R on get goes nowhere)
  int sees[2];
#pragma unroll
  for (int ri = 0; ri < 2; ++ri) {
    const int n = gid + 8 * ri;
    sees[ri] = w->k1 - w->k0 - (p.causal ? p.T - 1 - (n - p.T * (n * p.t_mul >> 16)) : 0);
  }
  bool ok = wwait(&bars->q_full, seg_i & 1);
  uint32_t qa[D / 16][4];
  if (ok) {
    const uint32_t q0 = smem_u32(sQ);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      ldsm_x4(q0 + sw_off((lane & 7) + 8 * ((lane >> 3) & 1), kk * 16 + 8 * (lane >> 4), C::CHUNK_BYTES), qa[kk][0],
              qa[kk][1], qa[kk][2], qa[kk][3]);
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(&bars->q_empty);
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  const int key_of = warp * 16;  // this warp's first key of a tile: its page, [d / 64][16 keys][128 bytes]
  constexpr int PAGE_BYTES = 16 * D * 2, PAGE_CHUNK = 16 * 128;
  uint32_t ks = gkv % KST, kl = gkv / KST, vs = gkv % VST, vl = gkv / VST;
  const int nt = w->nt;
#pragma unroll 1
  for (int x = 0; ok && x < nt; ++x) {
    if (!wwait(&bars->k_full[ks], kl & 1)) {
      ok = false;
      break;
    }
    const uint32_t k0 = smem_u32(sK + ks * C::KV_BYTES + warp * PAGE_BYTES);
    float s[2][4] = {}, odd[2][4] = {};  // two sums each, so that eight MMAs do not wait in a row
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int mi = lane >> 3;  // matrix of the four: (keys half, d half)
      uint32_t b00, b01, b10, b11;
      ldsm_x4(k0 + sw_off(8 * (mi >> 1) + (lane & 7), kk * 16 + 8 * (mi & 1), PAGE_CHUNK), b00, b01, b10, b11);
      mma_bf16_16816(kk & 1 ? odd[0] : s[0], qa[kk], b00, b01);
      mma_bf16_16816(kk & 1 ? odd[1] : s[1], qa[kk], b10, b11);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->k_empty[ks]);
    if (++ks == KST) {
      ks = 0;
      ++kl;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] += odd[e >> 2][e & 3];
    const int key0 = (w->x0 + x) * kPxTile + key_of;
    const int there = w->k1 - w->k0 - key0;  // keys of the item from this warp's first one on
    if (p.causal ? there < 16 + p.T - 1 : there < 16) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 8 * h + 2 * tig + (e & 1) >= sees[e >> 1]) s[h][e] = -INFINITY;
    }
    // two rows a thread; four neighbours share a row
    float alpha[2] = {1.f, 1.f};
#pragma unroll
    for (int ri = 0; ri < 2; ++ri) {
      if (ri == 1 && p.R <= 8) break;
      float mx = fmaxf(fmaxf(s[0][2 * ri], s[0][2 * ri + 1]), fmaxf(s[1][2 * ri], s[1][2 * ri + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[ri], mx * p.c);
      const float m_use = m_new == -INFINITY ? 0.f : m_new;
      alpha[ri] = ex2_approx(m[ri] - m_use);
      float sum = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float pv = ex2_approx(fmaf(s[h][2 * ri + e], p.c, -m_use));
          s[h][2 * ri + e] = pv;
          sum += pv;
        }
      l[ri] = l[ri] * alpha[ri] + sum;
      m[ri] = m_new;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= alpha[0];
        o[n][1] *= alpha[0];
        o[n][2] *= alpha[1];
        o[n][3] *= alpha[1];
      }
    }
    const uint32_t pa[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]), pack_bf16x2(s[1][0], s[1][1]),
                            pack_bf16x2(s[1][2], s[1][3])};
    if (!wwait(&bars->v_full[vs], vl & 1)) {
      ok = false;
      break;
    }
    // V rows past the item's end hold whatever the pool or an earlier tile left there, and
    // 0 * NaN is not 0: this thread's keys of the two halves, as masks of their fragments
    const uint32_t in_lo = (2 * tig < there ? 0xffffu : 0u) | (2 * tig + 1 < there ? 0xffff0000u : 0u);
    const uint32_t in_hi = (2 * tig + 8 < there ? 0xffffu : 0u) | (2 * tig + 9 < there ? 0xffff0000u : 0u);
    const uint32_t v0 = smem_u32(sV + vs * C::KV_BYTES + warp * PAGE_BYTES);
#pragma unroll
    for (int np = 0; np < D / 16; ++np) {
      const int mi = lane >> 3;  // (keys half, d half)
      uint32_t a, b, c, d;
      ldsm_x4_t(v0 + sw_off(8 * (mi & 1) + (lane & 7), np * 16 + 8 * (mi >> 1), PAGE_CHUNK), a, b, c, d);
      mma_bf16_16816(o[2 * np], pa, a & in_lo, b & in_hi);
      mma_bf16_16816(o[2 * np + 1], pa, c & in_lo, d & in_hi);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->v_empty[vs]);
    if (++vs == VST) {
      vs = 0;
      ++vl;
    }
  }
  gkv += nt;
  if (!ok) {
    record_error(p.err, FA_ERR_TIMEOUT, SITE_PX_SOFTMAX);
    bars->abort_flag = 1;
  }

  // ---- the end: the eight warps' rows joined
  float* part_o = reinterpret_cast<float*>(sQ + C::Q_BYTES);  // [8 warps][8 rows][D], no unit after a slim one is wide
  float* part_m = ex;                                         // [8 warps][16 rows]
  float* part_l = ex + 8 * 16;
#pragma unroll
  for (int ri = 0; ri < 2; ++ri) {
    float x = l[ri];
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    if (tig == 0) {
      // a score that is NaN may have left the maximum at -inf, which would weigh the row 0
      part_m[warp * 16 + gid + 8 * ri] = x != x ? INFINITY : m[ri];
      part_l[warp * 16 + gid + 8 * ri] = x;
    }
  }
  const bool whole = w->k0 == 0 && w->from_start() && w->to_end();
  const int part_row = w->part + kPxUnit * w->me, out_row = w->out;
  constexpr int COLS = D / 32;  // columns of a thread in the joined rows, a row to a warp
#pragma unroll 1
  for (int ri = 0; 8 * ri < p.R; ++ri) {
    if (ri == 1) {
      named_bar_sync(2, 256);  // the first eight rows have been read
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] = o[n][2];
        o[n][1] = o[n][3];
      }
    }
    // (columns are turned round by the row, so that eight rows fall on all banks)
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
      *reinterpret_cast<float2*>(part_o + (warp * 8 + gid) * D + ((n * 8 + 2 * tig) ^ ((gid & 3) << 3))) =
          make_float2(o[n][0], o[n][1]);
    if (ri == 0) {
      ok = vote_all(1, 256, ok);
      if (!ok) return false;
    } else {
      named_bar_sync(2, 256);
    }
    const int row = warp + 8 * ri, col = lane * COLS;
    if (row >= p.R) continue;
    float mw[8], m_all = -INFINITY;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      mw[k] = part_m[k * 16 + row];
      m_all = fmaxf(m_all, mw[k]);
    }
    const float m_use = m_all == -INFINITY ? 0.f : m_all;
    float sum = 0.f, acc[COLS];
#pragma unroll
    for (int c = 0; c < COLS; ++c) acc[c] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float f = ex2_approx(mw[k] - m_use);
      sum = fmaf(f, part_l[k * 16 + row], sum);
      const float* of = part_o + (k * 8 + warp) * D + (col ^ ((warp & 3) << 3));
#pragma unroll
      for (int c = 0; c < COLS; ++c) acc[c] = fmaf(f, of[c], acc[c]);
    }
    if (whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (NaN stays NaN)
      __nv_bfloat16* dst = p.o + static_cast<size_t>(out_row + row) * D + col;
      if constexpr (COLS == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
      else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
      if (p.lse && lane == 0) p.lse[out_row + row] = sum == 0.f ? -INFINITY : (m_all + log2f(sum)) * kLn2;
    } else {
      float* dst = p.part + ((col >> 3) * p.part_rows + part_row + row) * 8 + (col & 7);
      if constexpr (COLS == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      else
        *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
      if (lane == 0) p.part_ml[part_row + row] = make_float4(m_all, sum, sum, 0.f);
    }
  }
  if (threadIdx.x == 0 && w->from_start())
    p.desc[(static_cast<size_t>(p.B) + w->s0) * p.Hkv + w->kvh] = whole ? make_int2(kPxDone, 0) : make_int2(w->me << 16 | w->ctas, w->part);
  return true;
}

// A segment of a wide or narrow unit, by one of the two softmax slots: thread r has row r of the
// slot's tile, TMEM lane r. False: a wait ran out (in narrow units as all eight warps voted).
template <int D>
__device__ __forceinline__ bool px_rows(const PxParams& p, const volatile PxSeg* w, PxBars* bars, uint8_t* sV, float* ex,
                                        uint32_t& phases, uint32_t& gkv, uint64_t tmo) {
  using C = PxCfg<D>;
  constexpr int VST = C::V_STAGES;
  // The reference maximum m is raised only when a row's maximum climbs more than this above it;
  // until then the exponentials stay below 2^8 and carry one constant factor that O / l cancels.
  constexpr float kRescaleSlack = 8.f;
  // formed anew in each segment: kept over both kinds of segments these are spilled in their loops
  int tid = threadIdx.x;
  asm volatile("" : "+r"(tid));
  const int t = tid >> 7, r = tid & 127;
  const volatile int* abort_flag = &bars->abort_flag;
  const uint32_t tmem = *const_cast<const volatile uint32_t*>(&bars->tmem_base);
  const uint32_t lane_base = static_cast<uint32_t>(r & 96) << 16;
  const uint32_t tS = tmem + lane_base + t * C::SLOT_COLS;
  const uint32_t tO = tS + C::O_OFF;
  const float2 c2 = make_float2(p.c, p.c);
  bool ok = true;
  auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_lean(bar, parity, tmo, abort_flag));
  };
  // This thread's row of the segment: its sequence, and its place among the R; -1: none.
  auto row_of = [&](int& seq) -> int {
    int x = r;
    asm volatile("" : "+r"(x));
    const int tile = w->tile + (w->wide() ? t : 0);
    if (p.R <= kPxTile) {
      const int q = x * p.r_mul >> 16;  // x / R
      seq = w->s0 + tile * p.spt + q;
      return q < p.spt && seq < w->s0 + w->n ? x - q * p.R : -1;
    }
    const int q = tile / p.TS;
    seq = w->s0 + q;
    const int rr = (tile - q * p.TS) * kPxTile + x;
    return rr < p.R ? rr : -1;
  };
  const bool wide = w->wide();
  int sees = 0x7fffffff;  // keys that the row sees from the segment's first on; rows of nobody are not masked
  bool has_rows;
  {
    int seq;
    const int rr = row_of(seq);
    has_rows = __any_sync(0xffffffffu, rr >= 0);
    if (rr >= 0) {
      const int S = w->own() ? w->k1 : px_len(p, seq);
      const int pos = p.R <= kPxTile ? rr - p.T * (rr * p.t_mul >> 16) : rr % p.T;
      sees = min(p.causal ? S - p.T + pos + 1 : S, w->k1) - w->k0 - w->x0 * kPxTile;
    }
  }
  const int keys = w->k1 - w->k0 - w->x0 * kPxTile;  // of the item, from the segment's first one on
  const int nt = w->nt;
  const int x_first = wide ? 0 : t, step = wide ? 1 : 2;
  const int mine = wide ? nt : (nt - t + 1) / 2;  // tiles of this slot
  float m = -INFINITY;
  float l = 0.f;   // sum of the unrounded p: the lse's
  float lc = 0.f;  // bf16(p_top) - p_top of each tile's largest p, rescaled like l

#pragma unroll 1
  for (int i = 0; i < mine; ++i, phases ^= 1) {
    const int x = x_first + i * step;  // tile of the segment
    const int key0 = x * kPxTile;
    if (!wwait(&bars->s_full[t], phases & 1)) {
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
      if (__any_sync(0xffffffffu, sees < key0 + kPxTile)) {
        const int left = sees - key0;
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if (k >= left) s[k] = -INFINITY;
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
      const float alpha = sees == 0x7fffffff ? 1.f : ex2_approx(m - m_use);
      // the largest p is not 1 against a stale reference: O's normaliser counts it as the
      // bf16 product sees it, so that a nearly one-hot row is not off by its rounding
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
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o0[32];
          tmem_ld32(tO + cc * 32, o0);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 v0 = fmul2(make_float2(__uint_as_float(o0[k]), __uint_as_float(o0[k + 1])), al2);
            o0[k] = __float_as_uint(v0.x);
            o0[k + 1] = __float_as_uint(v0.y);
          }
          tmem_st32(tO + cc * 32, o0);
        }
      }
    }
    // V rows past the item's end hold whatever the pool or an earlier tile left there, and
    // 0 * NaN is not 0: the slot whose PV on this tile comes first zeroes them
    const int rows_there = keys - key0;
    if (rows_there < kPxTile && (!wide || t == 0)) {
      const uint32_t xg = gkv + x;
      if (!wwait(&bars->v_full[xg % VST], (xg / VST) & 1)) {
        ok = false;
        break;
      }
      uint8_t* vt = sV + (xg % VST) * C::KV_BYTES;
#pragma unroll 1
      for (int idx = r; idx < (kPxTile - rows_there) * C::KCH * 8; idx += 128) {
        const int vr = rows_there + idx / (C::KCH * 8);
        const int rem = idx % (C::KCH * 8);
        *reinterpret_cast<uint4*>(vt + (rem >> 3) * C::CHUNK_BYTES + vr * 128 + (rem & 7) * 16) =
            make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      __syncwarp();  // lanes may have made one store more than others, and what follows is the whole warp's
    }
    tmem_st_wait();
    tc_fence_before();
    mbar_arrive(&bars->p_full[t]);
  }
  gkv += nt;
  if (ok && mine > 0) {
    if (!wwait(&bars->pv_done[t], (phases >> 1) & 1)) ok = false;
    phases ^= 2;
    tc_fence_after();
  }

  // ---- the segment's end: final rows, or a partial
  int seq;
  const int rr = row_of(seq);
  const bool valid = rr >= 0;
  if (!valid) {
    m = -INFINITY;
    l = lc = 0.f;
  }
  // A score that is NaN (a query that is not finite) may have left m at -inf, which would
  // weigh the row 0: at +inf its weight, 2^(m - m), is NaN, here and in every join.
  if (l != l) m = INFINITY;
  const bool whole = w->own() && w->k0 == 0 && w->from_start() && w->to_end();
  float m_all = m, sum = l + lc, lsum = l;
  float f0 = 1.f, f1 = 0.f;  // weights of this slot's O (wide), or of slot 0's and slot 1's (narrow)
  if (!wide) {
    ex[t * 128 + r] = m;
    ex[(2 + t) * 128 + r] = l + lc;
    if (t == 1) ex[4 * 128 + r] = l;
    if (!ok) {
      record_error(p.err, FA_ERR_TIMEOUT, SITE_PX_SOFTMAX);
      bars->abort_flag = 1;
    }
    tc_fence_before();
    ok = vote_all(1, 256, ok);
    if (!ok) return false;  // all eight warps leave in the same segment
    tc_fence_after();  // the other slot's O, whose end its own warps waited for
    const float m0 = ex[r], m1 = ex[128 + r];
    m_all = fmaxf(m0, m1);
    const float m_use = m_all == -INFINITY ? 0.f : m_all;
    f0 = ex2_approx(m0 - m_use);
    f1 = ex2_approx(m1 - m_use);
    sum = f0 * ex[256 + r] + f1 * ex[384 + r];
    if (t == 0) lsum = f0 * l + f1 * ex[512 + r];
  }
  if (whole) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (NaN stays NaN)
    f0 *= inv;
    f1 *= inv;
  }
  if (has_rows) {
    // the row's place in its item's partials, and in the output
    const int at_row = p.units * p.R * w->s0 + (w->hu * w->n + seq - w->s0) * p.R + rr;
    const int kvh = w->kvh, place = kvh - w->hu * p.V;
    const long long base = (static_cast<long long>(w->own()) * p.V + place) * p.area;
    const long long part_row = base + at_row + static_cast<long long>(kPxUnit) * w->me;
    const size_t out_row = (static_cast<size_t>(seq) * p.Hkv + kvh) * p.R + rr;
    // narrow: each slot's warps write half the columns of the joined O
    const bool take0 = f0 != 0.f;
    const bool take1 = !wide && nt > 1 && f1 != 0.f;
    const uint32_t o_base = tmem + lane_base + (wide ? t * C::SLOT_COLS : 0) + C::O_OFF;
    const int c_lo = wide ? 0 : t * (D / 16), c_hi = wide ? D / 8 : c_lo + D / 16;  // chunks of eight columns
#pragma unroll 1
    for (int cc = c_lo; cc < c_hi; cc += 2) {  // (two at a time: a chunk's loads and stores one behind the other are 0.13 us)
      uint32_t a[2][8], b[2][8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        tmem_ld8(o_base + (cc + i) * 8, a[i]);
        tmem_ld8(o_base + (wide ? 0 : C::SLOT_COLS) + (cc + i) * 8, b[i]);
      }
      tmem_ld_wait();
      if (valid) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // TMEM that no PV wrote, and rows whose weight is 0 over whatever P held, are not taken in
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            o[k] = take0 ? f0 * __uint_as_float(a[i][k]) : 0.f;
            o[k] = take1 ? fmaf(f1, __uint_as_float(b[i][k]), o[k]) : o[k];
          }
          if (whole) {
            // (o may start on any 16-byte border)
            *reinterpret_cast<uint4*>(p.o + out_row * D + (cc + i) * 8) =
                make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
          } else {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(o[k]);
            st32(p.part + ((cc + i) * p.part_rows + part_row) * 8, v);
          }
        }
      }
      __syncwarp();  // lanes without a row wait: the next loads are the whole warp's
    }
    if (valid && (wide || t == 0)) {
      if (whole) {
        if (p.lse) p.lse[out_row] = lsum == 0.f ? -INFINITY : (m_all + log2f(lsum)) * kLn2;
      } else {
        p.part_ml[part_row] = make_float4(m_all, sum, lsum, 0.f);
      }
      if (w->from_start() && rr % kPxTile == 0) {  // this CTA begins the unit
        const size_t at = ((static_cast<size_t>(w->own()) * p.B + seq) * p.Hkv + kvh) * p.TS + rr / kPxTile;
        p.desc[at] = whole ? make_int2(kPxDone, 0) : make_int2(w->me << 16 | w->ctas, static_cast<int>(base + at_row));
      }
    }
  }
  tc_fence_before();
  return ok;
}

template <int D>
__global__ void __launch_bounds__(384, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKp,
                  const __grid_constant__ CUtensorMap tmVp, const PxParams p) {
  using C = PxCfg<D>;
  constexpr int KST = C::K_STAGES, VST = C::V_STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  PxBars* bars = reinterpret_cast<PxBars*>(smem + C::OFF_BAR);
  float* ex = reinterpret_cast<float*>(smem + C::OFF_EX);  // [5][128]: max and sum of both slots, lse sum of slot 1

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const int me = cta / p.V;  // this CTA's number on its line

  if (smem_u32(smem) & 1023u) {  // the swizzle atoms' alignment; the block's only shared memory starts at a multiple
    pdl_wait();
    if (threadIdx.x == 0) record_error(p.err, FA_ERR_TIMEOUT, SITE_PX_SMEM);
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 8);
#pragma unroll 1
    for (int s = 0; s < 6; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->k_empty[s], 8);
      mbar_init(&bars->v_empty[s], 8);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 128);
      mbar_init(&bars->pv_done[t], 1);
    }
    mbar_init(&bars->drain, 1);
    for (int e = 0; e < kPxQueue; ++e) {
      mbar_init(&bars->seg_full[e], 1);
      mbar_init(&bars->seg_empty[e], kPxReaders);
      bars->seg[e].nt = 0;
    }
    bars->abort_flag = 0;
    bars->it0 = bars->off0 = bars->group0 = 0;
    fence_barrier_init();
  }
  if (warp == 9) tmem_alloc(&bars->tmem_base, 512);

  // ---- this CTA's share of its line's cost: a block-wide scan over the items. Groups and lengths
  // go through shared memory that the rings use later: one round trip to L2 for all of them.
  // The walking warp is not in it: its code is on its way meanwhile.
  PxItem* item0 = reinterpret_cast<PxItem*>(ex + 128);  // what it begins in, until the walk has read it
  PxWalk* walk0 = reinterpret_cast<PxWalk*>(ex + 160);  // and how the line is cut
  if (warp != kPxWalker) {
    constexpr int kScan = kPxWalker * 32;
    PxWalk walk;
    pdl_wait();
    const int items = p.G + p.B;
    const int per = (items + kScan - 1) / kScan;
    const int lo = min(items, static_cast<int>(threadIdx.x) * per), hi = min(items, lo + per);
    int* gs = reinterpret_cast<int*>(sK);  // [G + 1]: starts
    int* gp = gs + p.G + 1;                // [G]: prefixes as they were asked for
    int* ls = gp + p.G;                    // [B]: lengths, where there is room for them
    const bool lens_here = p.B <= C::MOST_LENS;
#pragma unroll 1
    for (int i = threadIdx.x; i <= p.G; i += kScan) {
      gs[i] = __ldg(p.starts + i);
      if (i < p.G) gp[i] = __ldg(p.prefix_lens + i);
    }
    if (lens_here) {
#pragma unroll 1
      for (int i = threadIdx.x; i < p.B; i += kScan) ls[i] = px_len(p, i);
    }
    named_bar_sync(3, kScan);
    bool bad = false, wrong = false;  // the groups are not what they should be; seen by this thread
#pragma unroll 1
    for (int i = threadIdx.x; i < p.G; i += kScan) wrong |= gs[i] < 0 || gs[i] > gs[i + 1] || gs[i + 1] > p.B;
    auto len = [&](int b) { return lens_here ? ls[b] : px_len(p, b); };
    auto prefix_of = [&](int g) {
      const int s0 = gs[g], s1 = gs[g + 1];
      // (until the sums are made it is not known whether the starts are in order)
      return group_of_several(s0, s1, p.B) ? max(0, min(gp[g], len(s0))) & ~15 : 0;
    };
    auto item = [&](int i, int& g) {
      if (i < p.G) return bad ? PxItem{0, 0, 0, 0, 0, false} : px_group(p, gs[i], gs[i + 1], prefix_of(i));
      const int b = i - p.G;
      int prefix = 0;
      if (!bad) {
        if (g < 0) {  // the last that begins at or before b
          int top = p.G;
#pragma unroll 1
          for (g = 0; top - g > 1;) {
            const int mid = (g + top) / 2;
            if (gs[mid] <= b) g = mid; else top = mid;
          }
        }
#pragma unroll 1
        while (g + 1 < p.G && gs[g + 1] <= b) ++g;
        if (b >= gs[g] && b < gs[g + 1]) prefix = prefix_of(g);
      }
      return PxItem{b, b + 1, prefix, len(b), p.TS, true};
    };
    // Over the thread's items for the sums of steps and cost (a line's whole cost is below 2^31),
    // again where the groups turn out to be wrong; and, in the thread whose items hold the share's
    // start, where there are several, for the one that does.
    int4* wsum = reinterpret_cast<int4*>(ex);  // totals per warp, in the exchange area that nothing uses yet
    int off = -1, g;
    PxItem x = {0, 0, 0, 0, 0, false};
    walk.c = p.cost;
    while (true) {
      int steps = 0, mine = 0;
      g = -1;
#pragma unroll 1
      for (int i = lo; i < hi; ++i) {
        x = item(i, g);
        const int cost = x.head(walk.c) * p.units;
        if (off < 0) {
          steps += x.head(PX_BY_STEPS) * p.units;
          mine += cost;
        } else {
          if (off < cost) {
            bars->it0 = i;
            bars->off0 = off;
            bars->group0 = max(g, 0);
            *item0 = x;
            break;
          }
          off -= cost;
        }
      }
      if (off >= 0) break;
      int2 inc = make_int2(mine, steps);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc.x, o), z = __shfl_up_sync(0xffffffffu, inc.y, o);
        if (lane >= o) {
          inc.x += y;
          inc.y += z;
        }
      }
      const bool warp_wrong = __any_sync(0xffffffffu, wrong);
      if (lane == 31) wsum[warp] = make_int4(inc.x, inc.y, warp_wrong, 0);
      named_bar_sync(3, kScan);
      int2 before = make_int2(inc.x - mine, inc.y - steps), all = make_int2(0, 0);
      int any_wrong = 0;
#pragma unroll
      for (int w = 0; w < kPxWalker; ++w) {
        const int4 v = wsum[w];
        if (w < warp) {
          before.x += v.x;
          before.y += v.y;
        }
        all.x += v.x;
        all.y += v.y;
        any_wrong |= v.z;
      }
      if (any_wrong && !bad) {  // every sequence by itself then
        bad = true;
        if (threadIdx.x == 0) record_error(p.err, FA_ERR_BOUNDS, SITE_PX_GROUPS);
        named_bar_sync(3, kScan);
        continue;
      }
      const int grid = static_cast<int>(gridDim.x) / p.V;
      // Lines of so few steps that a CTA has hardly more than one are cut by steps alone. A share
      // is a step's cost or more either way, so that every CTA between a unit's first and last
      // has a step of it.
      int shares = grid;
      if (all.y <= 2 * grid) {
        walk.c = PX_BY_STEPS;
        before.x = before.y;
        mine = steps;
        all.x = all.y;
        shares = min(grid, max(1, all.y));
      }
      walk.cut = PxCut(all.x, shares);
      walk.no_groups = bad;
      walk.at = me < shares ? walk.cut.begin(me) : all.x;
      walk.end = me < shares ? walk.cut.begin(me + 1) : all.x;
      if (!(walk.at < walk.end && walk.at >= before.x && walk.at < before.x + mine)) break;
      off = walk.at - before.x;  // one thread
      if (hi - lo == 1) {
        bars->it0 = lo;
        bars->off0 = off;
        bars->group0 = max(g, 0);
        *item0 = x;
        break;
      }
    }
    if (threadIdx.x == 0) *walk0 = walk;
  }
  fence_async_smem();  // the rings' memory was read and written by plain accesses
  if (warp != kPxWalker) __syncthreads();
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
    if (warp == 8 || warp == 10) {
      // ======================= producers: K (and Q), V =======================
      const bool is_k = warp == 8;
      const CUtensorMap* my_map = is_k ? &tmK : &tmV;
      const CUtensorMap* my_pages = is_k ? &tmKp : &tmVp;  // slim: a page with all of d
      uint8_t* my_ring = is_k ? sK : sV;
      uint64_t* my_full = is_k ? bars->k_full : bars->v_full;
      uint64_t* my_empty = is_k ? bars->k_empty : bars->v_empty;
      const uint32_t ST = is_k ? KST : VST;
      if (lane == 0) {
        if (is_k) tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(my_map);
        tma_prefetch_desc(my_pages);
      }
      PxTake take;
      // one answer for all lanes, which go on or leave together
      auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_lean(bar, parity, tmo, abort_flag));
      };
      uint32_t g = 0;  // key tiles loaded so far (ring position)
      uint32_t stage = 0, lap = 0;
      uint32_t q_loads = 0;
      bool ok = true;
#pragma unroll 1
      while (__all_sync(0xffffffffu, ok && !*abort_flag)) {
        PxSeg w;
        {
          const volatile PxSeg* from = take.next(bars, tmo, abort_flag);
          if (!from) {
            ok = false;
            break;
          }
          w.s0 = from->s0;
          w.k0 = from->k0;
          w.k1 = from->k1;
          w.tile = from->tile;
          w.hu = from->hu;
          w.x0 = from->x0;
          w.nt = from->nt;
          w.flags = from->flags;
          w.kvh = from->kvh;
          take.done(bars);
        }
        if (w.nt == 0) break;
        const int* trow = p.block_table + static_cast<size_t>(w.s0) * p.max_pages;
        const int kvh = w.kvh;
        const bool slim = w.own() && p.R <= kPxSlim;
        const int page0 = w.k0 >> 4;  // (k0 is a page's start)
        const int n_pages = (w.k1 + 15) >> 4;
        // a lane holds one of 32 entries, four tiles' worth; the next 32 are fetched meanwhile
        auto fetch = [&](int x) -> int {
          const int pg = page0 + (w.x0 + x) * 8 + lane;
          return pg < n_pages && x * 8 + lane < w.nt * 8 ? __ldg(trow + pg) : -1;
        };
        int ent = -1, ent_next = fetch(0);
        // The last segment's Q is in use until its last S: this one's first tiles go ahead of
        // its Q (all but one stage of the ring, which that segment's own end frees).
        bool q_due = is_k;
        auto load_q = [&]() {
          if (lane == 0) {
            const int rows = min(p.R, kPxTile) * p.spt;  // of a box; those behind the batch's end are zeros
            const int tiles = w.wide() ? 2 : 1;
            mbar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(tiles * C::KCH * rows * 128));
#pragma unroll 1
            for (int t = 0; t < tiles; ++t) {
              const int tile = w.tile + t, seq = tile / p.TS;
              for (int c = 0; c < C::KCH; ++c)
                tma_load_4d(sQ + t * C::Q_BYTES + c * C::CHUNK_BYTES, &tmQ, &bars->q_full, c * 64,
                            (tile - seq * p.TS) * kPxTile, kvh, w.s0 + seq * p.spt);
            }
          }
          ++q_loads;
          q_due = false;
        };
        auto q_free = [&]() {
          return q_loads == 0 || __all_sync(0xffffffffu, mbar_test(&bars->q_empty, (q_loads - 1) & 1));
        };
#pragma unroll 1
        for (int x = 0; x < w.nt; ++x, ++g) {
          if (q_due) {
            if (q_free()) {
              load_q();
            } else if (x == KST - 1) {
              if (!wwait(&bars->q_empty, (q_loads - 1) & 1)) {
                ok = false;
                break;
              }
              load_q();
            }
          }
          if ((x & 3) == 0) {
            ent = ent_next;
            ent_next = fetch(x + 4);
          }
          const int npg = min(8, n_pages - page0 - (w.x0 + x) * 8);  // pages past the end are not loaded
          const int pi = slim ? lane : lane / C::KCH, pc = lane % C::KCH;  // the box of this lane: page and d-chunk
          int pe = __shfl_sync(0xffffffffu, ent, (x & 3) * 8 + (pi & 7));
          if (pi < npg && (pe < 0 || pe >= p.num_pages)) {
            // never dereferenced: page 0 is loaded in its place, the output is undefined
            record_error(p.err, FA_ERR_BOUNDS, SITE_PX_TABLE);
            pe = 0;
          }
          if (g >= ST && !wwait(&my_empty[stage], (lap & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&my_full[stage], static_cast<uint32_t>(npg) * 16 * 128 * C::KCH);
          __syncwarp();
          if (slim && pi < npg)
            tma_load_4d(my_ring + stage * C::KV_BYTES + pi * (16 * D * 2), my_pages, &my_full[stage], 0, kvh, pe * 16, 0);
          else if (pi < npg)
            tma_load_3d(my_ring + stage * C::KV_BYTES + pc * C::CHUNK_BYTES + pi * 2048, my_map, &my_full[stage], pc * 64,
                        kvh, pe * 16);
          if (++stage == ST) {
            stage = 0;
            ++lap;
          }
        }
        if (ok && q_due) {
          if (q_loads > 0 && !wwait(&bars->q_empty, (q_loads - 1) & 1))
            ok = false;
          else
            load_q();
        }
      }
      if (!ok) fail(SITE_PX_PRODUCER);
      // Copies in flight must land before the CTA exits. Waited for whether or not a wait has
      // run out so far: another role's may after this warp has issued its last copy.
      if (q_loads > 0) mbar_wait_lean(&bars->q_full, (q_loads - 1) & 1, tmo_unwind);
#pragma unroll 1
      for (uint32_t x = g > ST ? g - ST : 0; x < g; ++x) mbar_wait_lean(&my_full[x % ST], (x / ST) & 1, tmo_unwind);
    } else if (warp == 9) {
      // ======================= MMA issuer =======================
      const bool leader = elect_one();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kPxTile, 0, 0);
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
      const uint64_t dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = smem_desc_sw128(smem_u32(sV), C::CHUNK_BYTES, 1024);
      // S of slot t = Q (row tile q) K^T, K in ring stage st
      auto qk = [=](int t, int q, uint32_t st) {
        const uint64_t a0 = dQ + static_cast<uint64_t>((q * C::Q_BYTES) >> 4);
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
      auto pv = [=](int t, uint32_t st, bool first) {
        const uint64_t b0 = dV + static_cast<uint64_t>((st * C::KV_BYTES) >> 4);
        const uint32_t dO = tmem + t * C::SLOT_COLS + C::O_OFF;
        const uint32_t aP = tmem + t * C::SLOT_COLS;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kPxTile / 16; ++kk)
            tc_mma_ts(dO, aP + kk * 8, b0 + static_cast<uint64_t>((kk * 2048) >> 4), idesc_pv, (!first || kk > 0) ? 1u : 0u);
        }
      };
      auto commit = [=](uint64_t* bar) {
        if (leader) tc_commit(bar);
      };
      // what slim units free by eight warps' arrivals
      auto release = [=](uint64_t* bar) {
        if (leader) {
          mbar_arrive_n(bar, 7);
          tc_commit(bar);
        }
      };
      auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool { return mbar_wait_lean(bar, parity, tmo, abort_flag); };
      auto wait_k = [&](uint32_t x) -> bool {
        const bool r = wwait(&bars->k_full[x % KST], (x / KST) & 1);
        tc_fence_after();
        return r;
      };
      auto wait_v = [&](uint32_t x) -> bool {
        const bool r = wwait(&bars->v_full[x % VST], (x / VST) & 1);
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
      PxTake take;
      uint32_t g = 0;  // key tiles of earlier segments (ring position)
      bool ok = true;
#pragma unroll 1
      for (int nt; __all_sync(0xffffffffu, ok); g += nt) {  // (a wait may run out for some of the lanes only)
        const volatile PxSeg* from = take.next(bars, tmo, abort_flag);
        if (!from) {
          ok = false;
          break;
        }
        nt = from->nt;
        const bool wide = from->wide(), slim = from->own() && p.R <= kPxSlim;
        const uint32_t seg_i = take.i;
        take.done(bars);
        if (nt == 0) break;
        if (slim) continue;  // the softmax warps do those by themselves
        if (!wwait(&bars->q_full, seg_i & 1)) {
          ok = false;
          continue;
        }
        tc_fence_after();
        if (!wide) {
          // slots take the tiles in turn: tile x in slot x & 1
          auto score = [&](int x) -> bool {
            if (!wait_k(g + x)) return false;
            qk(x & 1, 0, (g + x) % KST);
            commit(&bars->s_full[x & 1]);
            release(&bars->k_empty[(g + x) % KST]);
            if (x + 1 == nt) release(&bars->q_empty);  // the segment's last S
            return true;
          };
          // the first two tiles' S, then PV of each with the S of the next but one right behind it:
          // that overwrites the columns P was read from, and one thread's MMAs run in order
#pragma unroll 1
          for (int x = -2; ok && x < nt; ++x) {
            if (x >= 0) {
              const int t = x & 1;
              if (!wait_p(t) || !wait_v(g + x)) {
                ok = false;
                break;
              }
              pv(t, (g + x) % VST, x < 2);
              release(&bars->v_empty[(g + x) % VST]);
              if (x + 2 >= nt) commit(&bars->pv_done[t]);
            }
            if (x + 2 < nt) ok = score(x + 2);
          }
        } else {
          // the first tile's S for both row tiles, then PV of each with the S of the next behind it
#pragma unroll 1
          for (int x = -1; ok && x < nt; ++x) {
            const uint32_t sv = (g + x) % VST, sk = (g + x + 1) % KST;
            const bool more = x + 1 < nt;
#pragma unroll 1
            for (int t = 0; t < 2; ++t) {
              if (x >= 0) {
                if (!wait_p(t) || (t == 0 && !wait_v(g + x))) {
                  ok = false;
                  break;
                }
                pv(t, sv, x == 0);
                if (t == 1) release(&bars->v_empty[sv]);
                if (!more) commit(&bars->pv_done[t]);
              }
              if (more) {
                if (t == 0 && !wait_k(g + x + 1)) {
                  ok = false;
                  break;
                }
                qk(t, t, sk);
                commit(&bars->s_full[t]);
              }
            }
            if (ok && more) {
              release(&bars->k_empty[sk]);
              if (x + 2 == nt) release(&bars->q_empty);
            }
          }
        }
      }
      if (!ok) fail(SITE_PX_MMA);
      commit(&bars->drain);  // every MMA must finish before TMEM is released
      mbar_wait_lean(&bars->drain, 0, tmo_unwind);
    } else {
      // ======================= the walk =======================
      // Lengths and groups come from L2 and a step of the walk takes some divisions, 0.9 us: one
      // warp does it ahead of the others, which take the segments from shared memory.
      // A first step, whose result nobody takes, brings its code from L2 while the others make the scan.
      PxWalk walk;
      walk.it = walk.off = walk.at = walk.g = 0;
      walk.end = 1;
      walk.cut = PxCut(2, 2);
      walk.no_groups = true;
      walk.c = PX_BY_STEPS;
      walk.first = item0 + 1;
      if (lane == 0) item0[1] = PxItem{0, 1, 0, 3 * kPxTile, 1, true};  // two steps: half of them each
      __syncwarp();
      bool ok = true;
      const int place = cta % p.V;
#pragma unroll 1
      for (int i = -1;; ++i) {
        if (i == 0) {
          pdl_wait();
          __syncthreads();
          walk = *walk0;
          walk.it = bars->it0;
          walk.off = bars->off0;
          walk.g = bars->group0;
          walk.first = item0;
          __syncwarp();
        }
        PxSeg w;
        const bool more = walk.next(p, me, w);
        if (more) {  // (here, since a division or two is a tenth of what a slim unit takes)
          w.kvh = w.hu * p.V + place;
          w.me = me;
          w.out = (w.s0 * p.Hkv + w.kvh) * p.R;
          w.part = static_cast<int>((p.V + place) * p.area) + (p.units * w.s0 + w.hu) * p.R;
        } else {
          w.nt = 0;
        }
        if (i < 0) {
          asm volatile("" ::"r"(w.nt), "r"(w.ctas), "r"(w.out), "r"(w.part), "r"(w.tile));
          continue;
        }
        const uint32_t e = static_cast<uint32_t>(i) % kPxQueue;
        if (i >= kPxQueue) {
          const uint64_t bound = px_bound(tmo, bars->seg[e].nt);  // the one that is still there is waited for
          if (!__all_sync(0xffffffffu, mbar_wait_lean(&bars->seg_empty[e], ((i / kPxQueue) & 1) ^ 1, bound, abort_flag))) {
            ok = false;
            break;
          }
        }
        if (lane == 0) {
          bars->seg[e] = w;
          mbar_arrive(&bars->seg_full[e]);
        }
        __syncwarp();
        if (!more) break;
      }
      if (!ok) fail(SITE_PX_WALK);
      // rows that a kind has no partials of: somebody has to say so
#pragma unroll 1
      for (int b = cta; b < p.B; b += gridDim.x) {
        int gb = 0, top = p.G;
#pragma unroll 1
        while (!walk.no_groups && top - gb > 1) {
          const int mid = (gb + top) / 2;
          if (__ldg(p.starts + mid) <= b) gb = mid; else top = mid;
        }
        const int prefix = walk.no_groups ? 0 : px_prefix_of(p, b, gb);
        const int n = p.Hkv * p.TS;
        const size_t at = static_cast<size_t>(b) * n;
        if (prefix == 0)
#pragma unroll 1
          for (int i = lane; i < n; i += 32) p.desc[at + i] = make_int2(0, 0);
        if (px_len(p, b) <= prefix)
#pragma unroll 1
          for (int i = lane; i < n; i += 32) p.desc[static_cast<size_t>(p.B) * n + at + i] = make_int2(0, 0);
      }
    }
  } else {
    // ======================= softmax: warps 0-3 (slot 0), 4-7 (slot 1) =======================
    warpgroup_reg_alloc<C::SOFTMAX_REGS>();
    bool ok = true;
    PxTake take;
    uint32_t phases = 0;  // parities of this slot's s_full (bit 0) and pv_done (bit 1)
    uint32_t gkv = 0;     // ring position at the segment's start
    const volatile PxSeg* w;
    // All eight warps go on or leave together. And both slots' O and the exchange area have been
    // read by all before the next segment overwrites them.
    auto next = [&]() -> bool {
      w = take.next(bars, tmo, abort_flag);
      if (!w) ok = false;
      if (!ok) fail(SITE_PX_SOFTMAX);
      ok = vote_all(1, 256, ok);
      return ok && w->nt > 0;
    };
    // The slim segments are a share's last ones. A loop of their own: in one with the others,
    // values of both are spilled, to memory that a busy L1 has no room for (64 sequences of 4096
    // keys: 186 us, 169 without).
    bool more;
#pragma unroll 1
    while ((more = next()) && !(w->own() && p.R <= kPxSlim)) {
      ok = px_rows<D>(p, w, bars, sV, ex, phases, gkv, tmo);
      take.done(bars);
    }
#pragma unroll 1
    for (; more; more = next()) {
      if (!px_slim<D>(p, w, bars, sQ, sK, sV, ex, take.i, gkv, tmo)) break;  // (as all eight warps voted)
      take.done(bars);
    }
    tc_fence_before();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partials of each row that is not written yet, of its prefix and of its own keys:
// lse = log2 sum 2^(m_s - m) l_s + m, O = sum 2^(m_s - m) O_s / sum 2^(m_s - m) l_s. Four rows
// to a warp: eight lanes read a line of the four, four such groups of lanes a line each. 1, 2,
// 4 or 8 warps take the rows' partials in turn, three or four of each in flight.
struct PxJoin {
  const float* part;
  const float4* part_ml;
  const int2* desc;
  __nv_bfloat16* o;
  float* lse;
  long long rows;  // B * Hkv * R
  int R, TS, per_kind;  // descriptors of a kind
  int grid;        // CTAs of a line
  long long part_rows;
};

template <int D, int WPR>
__global__ void __launch_bounds__(256) prefix_join_kernel(const PxJoin p) {
  constexpr int NV = D / 32, IN = D == 64 ? 4 : 3;  // a lane's vectors of four columns, partials in flight
  __shared__ float4 red[WPR > 1 ? 8 : 1][NV][32];
  __shared__ float red_ml[WPR > 1 ? 8 : 1][3][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();
  const int sub = warp % WPR, my = (lane & 7) >> 1, col = (lane >> 3) * 8 + (lane & 1) * 4;
  const long long row = (static_cast<long long>(blockIdx.x) * (8 / WPR) + warp / WPR) * 4 + my;
  int2 d[2] = {make_int2(kPxDone, 0), make_int2(kPxDone, 0)};
  long long r_in_tile = 0;
  if (row < p.rows) {
    const unsigned head = static_cast<unsigned>(row) / static_cast<unsigned>(p.R);
    const int rr = static_cast<int>(row - static_cast<long long>(head) * p.R);
    const size_t at = static_cast<size_t>(head) * p.TS + rr / kPxTile;
    d[0] = p.desc[at];
    d[1] = p.desc[static_cast<size_t>(p.per_kind) + at];
    r_in_tile = rr % kPxTile;
  }
  const bool todo = d[1].x != kPxDone;
  int count[2];
  long long at[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int first = d[k].x >> 16;
    count[k] = d[k].x & 0xffff;
    at[k] = d[k].y + r_in_tile + static_cast<long long>(kPxUnit) * first;
    // (after a wait that ran out a descriptor may be anything)
    if (!todo || first < 0 || first + count[k] > p.grid || at[k] < 0 ||
        at[k] + static_cast<long long>(kPxUnit) * count[k] >= p.part_rows + kPxUnit)
      count[k] = 0;
  }
  const int n = count[0] + count[1];
  float m = -INFINITY, s = 0.f, l = 0.f;
  float4 acc[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  // A partial whose maximum is +inf (its scores were NaN) makes all of them NaN; one of -inf
  // had no key that the row sees.
  auto add = [&](float m2, float s2, float l2, const float4* o2) {
    if (m2 == -INFINITY) return;
    const float mn = fmaxf(m, m2);
    const float fa = ex2_approx(m - mn), fb = ex2_approx(m2 - mn);
    s = s * fa + s2 * fb;
    l = l * fa + l2 * fb;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      acc[j] = make_float4(acc[j].x * fa + o2[j].x * fb, acc[j].y * fa + o2[j].y * fb, acc[j].z * fa + o2[j].z * fb,
                           acc[j].w * fa + o2[j].w * fb);
    m = mn;
  };
  for (int i0 = sub; i0 < n; i0 += WPR * IN) {
    float4 ml[IN], v[IN][NV];
#pragma unroll
    for (int k = 0; k < IN; ++k) {
      const int i = i0 + WPR * k;
      ml[k] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
      if (i < n) {
        const long long x = i < count[0] ? at[0] + static_cast<long long>(kPxUnit) * i
                                         : at[1] + static_cast<long long>(kPxUnit) * (i - count[0]);
        ml[k] = p.part_ml[x];
#pragma unroll
        for (int j = 0; j < NV; ++j)
          v[k][j] = *reinterpret_cast<const float4*>(p.part + ((4 * j + (lane >> 3)) * p.part_rows + x) * 8 + (lane & 1) * 4);
      }
    }
#pragma unroll
    for (int k = 0; k < IN; ++k) add(ml[k].x, ml[k].y, ml[k].z, v[k]);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) red[warp][j][lane] = acc[j];
    if (col == 0) {
      red_ml[warp][0][my] = m;
      red_ml[warp][1][my] = s;
      red_ml[warp][2][my] = l;
    }
    __syncthreads();
    if (sub == 0)
      for (int k = warp + 1; k < warp + WPR; ++k) {
        float4 v[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) v[j] = red[k][j][lane];
        add(red_ml[k][0][my], red_ml[k][1][my], red_ml[k][2][my], v);
      }
  }
  if (todo && sub == 0) {
    const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      *reinterpret_cast<uint2*>(p.o + row * D + 32 * j + col) =
          make_uint2(pack_bf16x2(acc[j].x * inv, acc[j].y * inv), pack_bf16x2(acc[j].z * inv, acc[j].w * inv));
    if (p.lse && col == 0) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct PxShape {
  int R, spt, TS, V, grid;  // grid: CTAs of a line
  long long area, desc;     // rows of partials of a place and kind, descriptors of a kind
  size_t part, ml, all;     // bytes
};

// How the problem is laid out on `sms` SMs; false: sizes that the call does not take.
static bool px_shape(int B, int Hq, int Hkv, int T, int max_pages, int d, int sms, PxShape& s) {
  const long long R = static_cast<long long>(Hq / Hkv) * T;
  if (d != 64 && d != 128) return false;
  if (R >= (1ll << 30) || B * R > (1ll << 30) / Hkv || sms > 32767) return false;
  if (static_cast<long long>(max_pages) * 16 > (1ll << 31) - 256) return false;  // (a key's index, rounded up to whole tiles, has 32 bits)
  s.R = static_cast<int>(R);
  s.spt = R <= kPxTile ? static_cast<int>(kPxTile / R) : 1;
  s.TS = static_cast<int>((R + kPxTile - 1) / kPxTile);
  // KV heads side by side, as many as fit: their keys lie beside one another in a page. Up to
  // 16, and groups that leave few SMs over.
  s.V = 1;
  for (int h = Hkv < 16 ? Hkv : 16; h >= 1; --h)
    if (Hkv % h == 0 && h <= sms && sms % h <= sms / 24) {
      s.V = h;
      break;
    }
  const long long units = Hkv / s.V, tiles = (static_cast<long long>(max_pages) * 16 + kPxTile - 1) / kPxTile;
  // steps of a line: a row tile of every sequence over all keys, of its prefix and of its own
  const long long rows = 2ll * B * s.TS * units;
  if (rows > (1ll << 31) / kPxMostCost / tiles) return false;  // (their cost has 32 bits)
  s.grid = static_cast<int>(rows * tiles < sms / s.V ? rows * tiles : sms / s.V);
  s.area = units * R * B + static_cast<long long>(kPxUnit) * s.grid;
  if (2 * s.V * s.area >= (1ll << 31)) return false;  // (as have the partials' rows)
  s.desc = static_cast<long long>(B) * Hkv * s.TS;
  s.part = static_cast<size_t>(2 * s.V * s.area) * d * 4;
  s.ml = static_cast<size_t>(2 * s.V * s.area) * 16;
  s.all = s.part + s.ml + static_cast<size_t>(2 * s.desc) * 8;
  return true;
}

template <int D>
static int launch_prefix(const CUtensorMap& tq, const CUtensorMap (&tk)[2], const CUtensorMap (&tv)[2], const PxParams& p,
                         const PxJoin& j, int grid, int sms, cudaStream_t stream) {
  using C = PxCfg<D>;
  auto kfn = prefix_kernel<D>;
  // the attribute holds for the life of the device's context: asked for once per device
  static std::atomic<unsigned long long> asked{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda_failure(e);
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(asked.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return record_cuda_failure(e);
    asked.fetch_or(bit, std::memory_order_relaxed);
  }
  const int rc = launch_dependent(kfn, dim3(grid), dim3(C::THREADS), C::SMEM, stream, tq, tk[0], tv[0], tk[1], tv[1], p);
  if (rc != FA_OK) return rc;
  // warps to four rows: as many as there are of some 24 an SM
  const long long warps = (j.rows + 3) / 4;
  int wpr = 8;
  while (wpr > 1 && warps * wpr > 24ll * sms) wpr >>= 1;
  const dim3 blocks(static_cast<unsigned>((warps * wpr + 7) / 8));
  if (wpr == 8) return launch_dependent(prefix_join_kernel<D, 8>, blocks, dim3(256), 0, stream, j);
  if (wpr == 4) return launch_dependent(prefix_join_kernel<D, 4>, blocks, dim3(256), 0, stream, j);
  if (wpr == 2) return launch_dependent(prefix_join_kernel<D, 2>, blocks, dim3(256), 0, stream, j);
  return launch_dependent(prefix_join_kernel<D, 1>, blocks, dim3(256), 0, stream, j);
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_prefix_workspace_bytes(int B, int Hq, int Hkv, int T, int max_pages, int d, int num_sms) {
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || max_pages < 1 || d < 1 || num_sms < 1 || Hq % Hkv != 0) return 0;
  PxShape s;
  return px_shape(B, Hq, Hkv, T, max_pages, d, num_sms, s) ? s.all : 0;
}

fa_status fa_prefix_decode_paged(const void* q, const void* k_pages, const void* v_pages, const int* block_table,
                                 const int* seqlens, const int* group_starts, const int* prefix_lens, int groups,
                                 void* o, float* lse, int B, int Hq, int Hkv, int T, int max_pages, int page_size,
                                 int num_pages, int d, float scale, int causal, void* workspace, size_t ws_bytes,
                                 void* stream) {
  auto mis = [](const void* x, uintptr_t m) { return (reinterpret_cast<uintptr_t>(x) & (m - 1)) != 0; };
  if (!q || !k_pages || !v_pages || !block_table || !seqlens || !group_starts || !prefix_lens || !o)
    return FA_ERR_INVALID_ARG;
  if (mis(q, 16) || mis(k_pages, 16) || mis(v_pages, 16) || mis(o, 16) || mis(block_table, 4) || mis(seqlens, 4) ||
      mis(group_starts, 4) || mis(prefix_lens, 4) || (lse && mis(lse, 4)) || mis(workspace, 256))
    return FA_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || T < 1 || max_pages < 1 || num_pages < 1 || groups < 1 || Hq % Hkv != 0 ||
      !(scale > 0.f) || !(scale < INFINITY))
    return FA_ERR_INVALID_ARG;
  if (page_size != 16 || (d != 64 && d != 128) || groups > FA_PREFIX_MAX_GROUPS) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(num_pages) * 16 >= (1ll << 31) ||
      static_cast<long long>(max_pages) * 16 > (1ll << 31) - 256 || static_cast<long long>(B) * Hq * T >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  {
    // o, lse and the workspace are written while other CTAs still read the rest
    const long long rows = static_cast<long long>(B) * Hq * T, q_bytes = rows * d * 2;
    const long long pool = 32ll * num_pages * Hkv * d, b4 = 4ll * B;
    const struct { const void* p; long long n; } out[] = {{o, q_bytes}, {lse, rows * 4}, {workspace, static_cast<long long>(ws_bytes)}},
        in[] = {{q, q_bytes}, {k_pages, pool}, {v_pages, pool}, {block_table, b4 * max_pages}, {seqlens, b4},
                {group_starts, 4ll * groups + 4}, {prefix_lens, 4ll * groups}};
    for (int i = 0; i < 3; ++i) {
      for (const auto& x : in)
        if (overlap(out[i].p, out[i].n, x.p, x.n)) return FA_ERR_INVALID_ARG;
      for (int k = 0; k < i; ++k)
        if (overlap(out[i].p, out[i].n, out[k].p, out[k].n)) return FA_ERR_INVALID_ARG;
    }
  }
  const int sms = device_sm_count();
  PxShape s;
  if (sms && !px_shape(B, Hq, Hkv, T, max_pages, d, sms, s)) return FA_ERR_UNSUPPORTED;
  if (!workspace) return FA_ERR_INVALID_ARG;  // (of 0 bytes, which may be null, for sizes that are not taken)
  if (!sms) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  if (ws_bytes < s.all) return FA_ERR_INVALID_ARG;
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return FA_ERR_CUDA;
  CUtensorMap tq, tk[2], tv[2];
  {
    // a KV head's R rows are dense; a box is the rows of a tile, of several sequences or of one
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)s.R, (cuuint64_t)Hkv, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)s.R * d * 2, (cuuint64_t)Hkv * s.R * d * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)(s.R < kPxTile ? s.R : kPxTile), 1, (cuuint32_t)s.spt};
    cuuint32_t es[4] = {1, 1, 1, 1};
    if (enc(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(q), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return static_cast<fa_status>(record_cuda_failure(cudaErrorInvalidValue));
  }
  for (int i = 0; i < 4; ++i) {
    // K, V: one 16-token page of one KV head per box, 64 of its d (what a tile of 128 rows is made
    // of), or all of it (what a warp of a slim unit takes: half the boxes at d = 128). L2 fetches
    // what a row is, no neighbour's.
    const bool pages = i & 2;
    const CUtensorMapL2promotion fetch = d == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    cuuint64_t dims[4] = {(cuuint64_t)(pages ? 64 : d), (cuuint64_t)Hkv, (cuuint64_t)num_pages * 16, (cuuint64_t)d / 64};
    cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)Hkv * d * 2, 128};
    cuuint32_t box[4] = {64, 1, 16, (cuuint32_t)d / 64};
    cuuint32_t es[4] = {1, 1, 1, 1};
    if (enc(i & 1 ? &tv[i >> 1] : &tk[i >> 1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, pages ? 4 : 3,
            const_cast<void*>(i & 1 ? v_pages : k_pages), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, fetch, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return static_cast<fa_status>(record_cuda_failure(cudaErrorInvalidValue));
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PxParams p = {};
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.starts = group_starts;
  p.prefix_lens = prefix_lens;
  p.B = B;
  p.G = groups;
  p.Hkv = Hkv;
  p.T = T;
  p.R = s.R;
  p.causal = causal ? 1 : 0;
  p.spt = s.spt;
  p.TS = s.TS;
  p.r_mul = (1 << 16) / s.R + 1;
  p.t_mul = (1 << 16) / T + 1;
  p.V = s.V;
  p.units = Hkv / s.V;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.c = scale * kLog2e;
  // In eighths of a wide step (some 0.2 us); narrow and slim steps are two tiles of keys, which
  // at d = 128 wait for HBM. What a unit costs beside its steps: Q and the first S, a slim one's
  // join, the partials of 128 or 256 rows. Swept one or two at a time over batches from 10 to 170 us:
  // on 84 drawn ones 0.8 % on average from the best of 20 to 30 others for each, 8 % at most.
  p.cost = d == 128 ? PxCost{9, 16, 8, 20, 10, 9} : PxCost{9, 16, 8, 20, 8, 15};
  if (s.R <= kPxSlim) {
    p.cost.own_step = d == 128 ? 7 : 6;
    p.cost.own_front = d == 128 ? 4 : 6;
    p.cost.wide_front = d == 128 ? 4 : 12;
  }
  p.area = s.area;
  p.part_rows = 2 * s.V * s.area;
  p.part = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float4*>(ws + s.part);
  p.desc = reinterpret_cast<int2*>(ws + s.part + s.ml);
  p.err = device_error_word();
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  p.timeout_ns = wait_timeout_ns();
  const PxJoin j = {p.part, p.part_ml, p.desc, p.o, lse, static_cast<long long>(B) * Hkv * s.R, s.R, s.TS,
                    static_cast<int>(s.desc), s.grid, 2 * s.V * s.area};
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return static_cast<fa_status>(d == 128 ? launch_prefix<128>(tq, tk, tv, p, j, s.V * s.grid, sms, cs)
                                         : launch_prefix<64>(tq, tk, tv, p, j, s.V * s.grid, sms, cs));
}

}  // extern "C"
