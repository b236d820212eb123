// rope.cu -- rotary positions, forward and backward, and the same on the way into a
// paged K/V cache.
//
// Pair i of a row at position p, (a, b), becomes
//   (a cos t - b sin t, b cos t + a sin t) * mscale,  t = p * inv_freq[i];
// the gradient is the transpose, the same with -t. Pairs are (x[i], x[i + rot/2])
// ("half") or (x[2i], x[2i+1]) ("interleaved"), i < rot/2; values from rot on pass
// through.
//
// Angles. A far position needs t to a small part of 2 pi, which p * inv_freq in 32
// bits has not (at p = 10^6 it is off by 0.06). Here inv_freq / (2 pi) is a 64-bit
// fraction of a turn, so the integer product p * that, modulo 2^64, IS the angle
// modulo a turn, off by less than |p| * 2^-63 turns. What it is past the nearest quarter
// turn goes to sincospif.
// An inv_freq that is NaN, infinite or 2^53 and more makes its pairs NaN.
// No table of cosines, no largest position, no FP64 pipe (which is narrow here).
//
// How: bound by reading and writing each value once. A lane owns VEC pairs of a token
// (16 bytes on each side of a row); a block owns 32 such token-lanes and a chunk of the
// heads, one head to a warp at a time. The block makes the sines of its 32 token-lanes
// once (VEC angles to a warp, shared memory) while the first U rows of every warp are
// already on their way. A row's d * 2 bytes are whole 128-byte lines for the layouts
// that matter, whatever the strides between rows, so no transpose through shared memory
// is needed to go between [B][T][heads][d] and [B][heads][T][d]. b4 h16+16 n4096 d128: bf16
// 42 us, fp32 79 us (6.3 and 6.8 TB/s).
// Rows that are not whole aligned 16-byte vectors take the widest that they are, one width for
// the whole row (b4 h32 n4096 d72, 20 of them rotated, bf16: pairs of values, as its half of 10
// allows, 44 us, where the bytes take 22; single ones 79 us).
#include <math.h>

#include <initializer_list>
#include <type_traits>

#include "launch.cuh"
#include "rows.h"

namespace fa {

// One operand: rows [b][h][t], `heads` of them a token, strides in elements.
struct RopeSide {
  const void* src;
  void* dst;
  long long sb, sh, st;  // source strides
  long long db, dh, dt;  // destination strides (unused where rows go to slots)
  int heads;
};

struct RopeParams {
  RopeSide q, k, v;         // v.heads = 0 but for appends
  const int* positions;
  long long pos_sb;         // 0: one row of positions for the whole batch
  const double* inv_freq;
  const int* slots;         // appends: k and v rows go to slot * slot_stride + head * d
  long long slot_stride;
  int num_slots;
  long long tokens;         // B * T
  int T, d, rot, lanes, head_chunk;
  bool small;
  float mscale, sign;       // sign -1: the transposed rotation
  unsigned* err;
};

template <typename E>
struct Vec16;
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
};
template <>
struct Vec16<float> {
  static constexpr int N = 4;
};

// VEC values as they lie in memory (2 to 16 bytes, one access), and as floats
template <typename E, int VEC>
struct Raw {
  static constexpr int BYTES = VEC * sizeof(E);
  using T = typename std::conditional<
      BYTES == 16, uint4,
      typename std::conditional<BYTES == 8, uint2, typename std::conditional<BYTES == 4, uint32_t, E>::type>::type>::type;
  T r;
  __device__ __forceinline__ void load(const E* p) { r = *reinterpret_cast<const T*>(p); }
  __device__ __forceinline__ void store(E* p) const { *reinterpret_cast<T*>(p) = r; }
  __device__ __forceinline__ uint32_t word(int i) const {
    if constexpr (BYTES == 16)
      return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
    else if constexpr (BYTES == 8)
      return i == 0 ? r.x : r.y;
    else
      return r;
  }
  __device__ __forceinline__ void get(float (&v)[VEC]) const {
    if constexpr (BYTES == 2) {
      v[0] = static_cast<float>(r);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        v[i] = sizeof(E) == 4 ? __uint_as_float(word(i % (BYTES / 4)))
                              : __uint_as_float(i % 2 ? word(i / 2) & 0xffff0000u : word(i / 2) << 16);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[VEC]) {
    if constexpr (BYTES == 2) {
      r = static_cast<E>(v[0]);
    } else {
      uint32_t w[BYTES / 4];
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i)
        w[i] = sizeof(E) == 4 ? __float_as_uint(v[i % VEC]) : pack_bf16x2(v[2 * i % VEC], v[(2 * i + 1) % VEC]);
      if constexpr (BYTES == 16)
        r = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (BYTES == 8)
        r = make_uint2(w[0], w[1]);
      else
        r = w[0];
    }
  }
};

// f / (2 pi) modulo 1 as a 64-bit fraction, off by less than 2^-63 turns, from the double's bits:
// f = m * 2^-s with a 53-bit m, so the fraction is m * floor(2^128 / (2 pi)) shifted right by
// s + 64, modulo 2^64 (the constant loses less than |f| * 2^-128 turns, the shift 2^-64). False:
// f is NaN, infinite or not below 2^53.
__device__ __forceinline__ bool turns_of(double f, unsigned long long& turns) {
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(f));
  const int e = static_cast<int>((bits >> 52) & 0x7ff);
  const int s = 1075 - e;
  turns = 0;
  if (s < 0) return false;
  if (e == 0 || s >= 128) return true;  // zero, or far below 2^-64 turns
  const unsigned long long m = (bits & 0xfffffffffffffull) | (1ull << 52);
  constexpr unsigned long long kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;  // 1 / (2 pi), 128 bits
  const unsigned long long low = __umul64hi(m, kLo), mid = m * kHi + low;  // the product but its last 64 bits
  const unsigned long long top = __umul64hi(m, kHi) + (mid < low);
  const unsigned long long r = s < 64 ? (mid >> s) | (top << 1 << (63 - s)) : top >> (s - 64);
  turns = (bits >> 63) ? 0ull - r : r;
  return true;
}

constexpr int kRopeWarps = 8;
constexpr int kRopeMostRows = 4;  // of a warp

// U: rows of a warp, all in flight at once. The sines stay in shared memory: in registers
// they would cost a block's worth of occupancy (64 registers a thread: four blocks an SM;
// b1 hq64 hkv8 n8192 d128 52.9 us with them there, 47.2 us without).
template <typename E, int VEC, bool INTER, bool APPEND, int U>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_kernel(const RopeParams p) {
  __shared__ float cs[2][VEC][32];
  pdl_wait();
  pdl_launch();
  const int warp = threadIdx.x >> 5, id = threadIdx.x & 31;
  const long long at = static_cast<long long>(blockIdx.x) * 32 + id;  // this thread's token-lane
  // 32-bit division where the launch has fewer of them than 2^31
  const long long token = p.small ? static_cast<long long>(static_cast<unsigned>(at) / static_cast<unsigned>(p.lanes))
                                  : at / p.lanes;
  const int lane = static_cast<int>(at - token * p.lanes);
  const bool there = token < p.tokens;
  const int b = there ? static_cast<int>(static_cast<unsigned>(token) / static_cast<unsigned>(p.T)) : 0;
  const int t = there ? static_cast<int>(token - static_cast<long long>(b) * p.T) : 0;
  const int half = p.rot / 2;
  // A lane's two vectors lie half the part's length apart (in the rotated part, and in the
  // tail that it copies), so that neighbouring lanes' accesses are neighbours in memory.
  const int turning = half / VEC;       // lanes of the rotated part
  const bool turn = lane < turning;
  constexpr bool ADJ = INTER && VEC == 1;  // a pair is two neighbours, and a vector is one of them
  const int o0 = turn ? (ADJ ? 2 * lane : lane * VEC) : p.rot + (lane - turning) * VEC;
  const int o1 = turn ? (ADJ ? o0 + 1 : o0 + half) : o0 + (p.lanes - turning) * VEC;
  const bool two = turn || o1 < p.d;
  const int hq = p.q.heads, hk = hq + p.k.heads;
  const int h_begin = blockIdx.y * p.head_chunk;
  const int h_end = min(h_begin + p.head_chunk, hk + p.v.heads);

  long long slot = 0;
  if (APPEND && there && h_end > hq) {
    slot = __ldg(p.slots + token);
    if (slot < -1 || slot >= p.num_slots) {
      record_error(p.err, FA_ERR_BOUNDS, SITE_APPEND);
      slot = -1;
    }
  }
  // the operand of head h (the same for a whole warp) and the row's place in it
  auto side_of_head = [&](int h) -> const RopeSide& { return h < hq ? p.q : (h < hk ? p.k : p.v); };
  auto head_in_side = [&](int h) { return h < hq ? h : (h < hk ? h - hq : h - hk); };
  auto wanted = [&](int h) { return there && h < h_end && !(APPEND && h >= hq && slot < 0); };

  Raw<E, VEC> x[U], y[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h_begin + warp + u * kRopeWarps;
    if (wanted(h)) {
      const RopeSide& s = side_of_head(h);
      const E* src = static_cast<const E*>(s.src) + b * s.sb + head_in_side(h) * s.sh + t * s.st;
      x[u].load(src + o0);
      if (two) y[u].load(src + o1);
    }
  }

  if (turn && there) {
    const long long pos = __ldg(p.positions + b * p.pos_sb + t);
    for (int e = warp; e < VEC; e += kRopeWarps) {
      // interleaved: half of the lane's pairs are in its first vector, half in its second
      const int pair = !INTER || ADJ ? lane * VEC + e
                                     : (2 * e < VEC ? o0 / 2 + e : o1 / 2 + e - VEC / 2);
      unsigned long long a;
      const bool angle = turns_of(__ldg(p.inv_freq + pair), a);
      a *= static_cast<unsigned long long>(pos);
      // The nearest quarter turn comes off the whole number, so that rounding to 24 bits is
      // by 2^-24 of at most an eighth of a turn, as the sine and cosine of it need.
      const unsigned quarter = static_cast<unsigned>((a + (1ull << 61)) >> 62);
      const long long rest = static_cast<long long>(a - (static_cast<unsigned long long>(quarter) << 62));
      float s, c;
      sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);  // (in half turns)
      if (quarter & 1) {
        const float was = s;
        s = c;
        c = -was;
      }
      if (quarter & 2) {
        s = -s;
        c = -c;
      }
      if (!angle) s = c = NAN;
      cs[0][e][id] = c * p.mscale;
      cs[1][e][id] = s * p.mscale * p.sign;
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h_begin + warp + u * kRopeWarps;
    if (!wanted(h)) continue;
    const RopeSide& side = side_of_head(h);
    const bool to_slot = APPEND && h >= hq;
    if (turn && h < hk) {
      float xv[VEC], yv[VEC];
      x[u].get(xv);
      y[u].get(yv);
      // the pair's two values: element e of x and of y, or neighbours 2e, 2e + 1 of x, then y
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        float& a = !INTER ? xv[e] : (2 * e < VEC ? xv[(2 * e) % VEC] : yv[(2 * e) % VEC]);
        float& g = !INTER ? yv[e] : (2 * e + 1 < VEC ? xv[(2 * e + 1) % VEC] : yv[(2 * e + 1) % VEC]);
        const float a0 = a, g0 = g, c = cs[0][e][id], s = cs[1][e][id];
        a = a0 * c - g0 * s;
        g = g0 * c + a0 * s;
      }
      x[u].set(xv);
      y[u].set(yv);
    }
    const long long hs = head_in_side(h);
    E* dst = static_cast<E*>(side.dst) +
             (to_slot ? slot * p.slot_stride + hs * p.d : b * side.db + hs * side.dh + t * side.dt);
    x[u].store(dst + o0);
    if (two) y[u].store(dst + o1);
  }
}

// Whether every row of the operand starts on a border of `vec` values of `elem` bytes.
static bool rows_on(const RopeSide& s, int vec, unsigned elem, bool slots) {
  auto whole = [vec](long long x) { return x % vec == 0; };
  return whole(s.sb) && whole(s.sh) && whole(s.st) && (slots || (whole(s.db) && whole(s.dh) && whole(s.dt))) &&
         ((reinterpret_cast<uintptr_t>(s.src) | reinterpret_cast<uintptr_t>(s.dst)) & (vec * elem - 1)) == 0;
}

template <typename E, int VEC, bool APPEND>
static int launch_rope_rows(const RopeParams& p, bool interleaved, int rows, dim3 grid, cudaStream_t stream) {
  const dim3 block(kRopeWarps * 32);
  auto go = [&](auto inter, auto u) {
    return launch_dependent(rope_kernel<E, VEC, decltype(inter)::value, APPEND, decltype(u)::value>, grid, block, 0,
                            stream, p);
  };
  auto with = [&](auto inter) {
    if constexpr (VEC == Vec16<E>::N) {
      if (rows == 1) return go(inter, std::integral_constant<int, 1>{});
      if (rows == 2) return go(inter, std::integral_constant<int, 2>{});
      if (rows == 3) return go(inter, std::integral_constant<int, 3>{});
    }
    return go(inter, std::integral_constant<int, kRopeMostRows>{});
  };
  return interleaved ? with(std::true_type{}) : with(std::false_type{});
}

template <typename E, bool APPEND>
static int launch_rope(RopeParams& p, bool interleaved, cudaStream_t stream) {
  constexpr int V = Vec16<E>::N;
  // the widest vectors that are whole on both sides of every pair, in the tail and at every row's start
  int w = V;
  while (w > 1 && !((p.rot / 2) % w == 0 && p.d % w == 0 && rows_on(p.q, w, sizeof(E), false) &&
                    (p.k.heads == 0 || rows_on(p.k, w, sizeof(E), APPEND)) &&
                    (p.v.heads == 0 || rows_on(p.v, w, sizeof(E), true))))
    w /= 2;
  p.lanes = p.rot / 2 / w + ((p.d - p.rot) / w + 1) / 2;
  const int heads = p.q.heads + p.k.heads + p.v.heads;
  const long long blocks = (p.tokens * p.lanes + 31) / 32;
  if (blocks >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  p.small = blocks * 32 < (1ll << 31);
  // Heads of a block: up to four rows to each of its eight warps (a warp's heads are
  // kRopeWarps apart), in even cuts; fewer where the blocks would leave SMs idle (a decode
  // step).
  int cuts = (heads + kRopeMostRows * kRopeWarps - 1) / (kRopeMostRows * kRopeWarps);
  const int most = (heads + kRopeWarps - 1) / kRopeWarps;
  while (cuts < most && blocks * cuts < 2ll * device_sm_count()) cuts = cuts * 2 < most ? cuts * 2 : most;
  const int rows = ((heads + cuts - 1) / cuts + kRopeWarps - 1) / kRopeWarps;
  p.head_chunk = rows * kRopeWarps;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + p.head_chunk - 1) / p.head_chunk));
  if (w == V) return launch_rope_rows<E, V, APPEND>(p, interleaved, rows, grid, stream);
  if (V > 4 && w == 4) return launch_rope_rows<E, 4, APPEND>(p, interleaved, rows, grid, stream);
  if (w == 2) return launch_rope_rows<E, 2, APPEND>(p, interleaved, rows, grid, stream);
  return launch_rope_rows<E, 1, APPEND>(p, interleaved, rows, grid, stream);
}

static bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// The stride of a dimension of one is never used; callers leave anything there.
static RopeSide side_of(const void* src, void* dst, const long long* s, const long long* d, int B, int heads, int T) {
  RopeSide r = {};
  r.src = src;
  r.dst = dst;
  r.heads = heads;
  r.sb = B > 1 ? s[0] : 0;
  r.sh = heads > 1 ? s[1] : 0;
  r.st = T > 1 ? s[2] : 0;
  if (d) {
    r.db = B > 1 ? d[0] : 0;
    r.dh = heads > 1 ? d[1] : 0;
    r.dt = T > 1 ? d[2] : 0;
  }
  return r;
}

static Rows rows_of(const void* at, long long sb, long long sh, long long st, int B, int heads, int T, int d,
                    unsigned elem) {
  return Rows{at, {sb * elem, sh * elem, st * elem}, {B, heads, T}, static_cast<long long>(d) * elem};
}

// Whether a row of an output lies on one of another operand, or on another of its own: rows
// would be written that others still read. In place (a destination that is its source, stride
// for stride) is fine.
static bool outputs_meet(const RopeSide& q, const RopeSide& k, int B, int T, int d, unsigned elem,
                         const int* positions, long long pos_bytes, const double* inv_freq, long long freq_bytes) {
  auto src = [&](const RopeSide& s) { return rows_of(s.src, s.sb, s.sh, s.st, B, s.heads, T, d, elem); };
  auto dst = [&](const RopeSide& s) { return rows_of(s.dst, s.db, s.dh, s.dt, B, s.heads, T, d, elem); };
  auto in_place = [](const RopeSide& s) { return s.src == s.dst && s.sb == s.db && s.sh == s.dh && s.st == s.dt; };
  auto bad = [&](const RopeSide& s) {
    return (!in_place(s) && rows_meet(src(s), dst(s))) || rows_meet_themselves(dst(s)) ||
           rows_meet(dst(s), dense_rows(positions, pos_bytes)) || rows_meet(dst(s), dense_rows(inv_freq, freq_bytes));
  };
  return bad(q) || (k.heads > 0 && (bad(k) || rows_meet(dst(q), dst(k)) || rows_meet(dst(q), src(k)) ||
                                    rows_meet(src(q), dst(k))));
}

// Whether the rows of a source or of a destination meet `bytes` bytes at `at`, by the range that
// they span.
static bool span_meets(const void* rows, long long sb, long long sh, long long st, int B, int heads, int T, int d,
                      unsigned elem, const void* at, long long bytes) {
  long long lo = 0, hi = d;
  for (const long long reach : {sb * (B - 1), sh * (heads - 1), st * (T - 1)}) (reach < 0 ? lo : hi) += reach;
  return overlap(static_cast<const char*>(rows) + lo * elem, (hi - lo) * elem, at, bytes);
}

static fa_status check_rope(const void* q, const void* q_out, const int* positions, const double* inv_freq, int B,
                            int Hq, int Hk, int T, int d, int rot_dim, float mscale, unsigned elem) {
  if (!q || !q_out || !positions || !inv_freq) return FA_ERR_INVALID_ARG;
  if (misaligned(q, elem) || misaligned(q_out, elem) || misaligned(positions, 4) || misaligned(inv_freq, 8))
    return FA_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hk < 0 || T < 1 || d < 2 || rot_dim < 2 || (rot_dim & 1) || rot_dim > d)
    return FA_ERR_INVALID_ARG;
  if (!isfinite(mscale) || mscale <= 0.f) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * T >= (1ll << 31) || d > 1024 || Hq > 65535 || Hk > 65535) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

static fa_status rope_any(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
                          const int* positions, int positions_shared, const double* inv_freq, int B, int Hq, int Hk,
                          int T, int d, int rot_dim, int interleaved, float mscale, int dtype, float sign,
                          void* stream) {
  if (dtype != FA_DTYPE_BF16 && dtype != FA_DTYPE_F32) return FA_ERR_UNSUPPORTED;
  const unsigned elem = dtype == FA_DTYPE_F32 ? 4 : 2;
  const fa_status st = check_rope(q, q_out, positions, inv_freq, B, Hq, Hk, T, d, rot_dim, mscale, elem);
  if (st != FA_OK) return st;
  if (!strides || (Hk > 0 && (!k || !k_out || misaligned(k, elem) || misaligned(k_out, elem))))
    return FA_ERR_INVALID_ARG;
  RopeParams p = {};
  p.q = side_of(q, q_out, strides, strides + 3, B, Hq, T);
  if (Hk > 0) p.k = side_of(k, k_out, strides + 6, strides + 9, B, Hk, T);
  if (outputs_meet(p.q, p.k, B, T, d, elem, positions, 4ll * T * (positions_shared ? 1 : B), inv_freq, 4ll * rot_dim))
    return FA_ERR_INVALID_ARG;
  p.positions = positions;
  p.pos_sb = positions_shared ? 0 : T;
  p.inv_freq = inv_freq;
  p.tokens = static_cast<long long>(B) * T;
  p.T = T;
  p.d = d;
  p.rot = rot_dim;
  p.mscale = mscale;
  p.sign = sign;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int rc = dtype == FA_DTYPE_F32 ? launch_rope<float, false>(p, interleaved != 0, cs)
                                       : launch_rope<__nv_bfloat16, false>(p, interleaved != 0, cs);
  return static_cast<fa_status>(rc);
}

}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rope_inv_freq(double* inv_freq, float* mscale, int rot_dim, double base, int scaling, double factor,
                           double original_len, double beta_fast, double beta_slow) {
  if (!inv_freq || !mscale) return FA_ERR_INVALID_ARG;
  if (rot_dim < 2 || (rot_dim & 1) || !isfinite(base) || base <= 1.0) return FA_ERR_INVALID_ARG;
  if (scaling < FA_ROPE_PLAIN || scaling > FA_ROPE_YARN) return FA_ERR_UNSUPPORTED;
  if (scaling != FA_ROPE_PLAIN && (!isfinite(factor) || factor < 1.0)) return FA_ERR_INVALID_ARG;
  const int n = rot_dim / 2;
  const double two_pi = 6.283185307179586476925;
  *mscale = 1.f;
  // the base that stretches the longest wave by `factor` and leaves the shortest alone
  const double b = scaling == FA_ROPE_NTK && n > 1 ? base * pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2)) : base;
  double low = 0.0, high = 0.0;
  if (scaling == FA_ROPE_YARN) {
    if (!isfinite(original_len) || original_len < 1.0 || !isfinite(beta_fast) || !isfinite(beta_slow) ||
        beta_slow <= 0.0 || beta_fast < beta_slow)
      return FA_ERR_INVALID_ARG;
    // the (fractional) pair index whose wave turns r times within the original length
    auto pair_of = [&](double r) { return rot_dim * log(original_len / (r * two_pi)) / (2.0 * log(base)); };
    low = floor(pair_of(beta_fast));
    high = ceil(pair_of(beta_slow));
    if (low < 0.0) low = 0.0;
    if (high > rot_dim - 1) high = rot_dim - 1;
    if (high <= low) high = low + 0.001;
    if (factor > 1.0) *mscale = static_cast<float>(0.1 * log(factor) + 1.0);
  }
  for (int i = 0; i < n; ++i) {
    double f = pow(b, -2.0 * i / rot_dim);
    if (scaling == FA_ROPE_LINEAR) f /= factor;
    if (scaling == FA_ROPE_YARN) {
      double ramp = (i - low) / (high - low);  // 0: keeps its frequency, 1: stretched by `factor`
      ramp = ramp < 0.0 ? 0.0 : (ramp > 1.0 ? 1.0 : ramp);
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    inv_freq[i] = f;
  }
  return FA_OK;
}

fa_status fa_rope(const void* q, const void* k, void* q_out, void* k_out, const long long* strides,
                  const int* positions, int positions_shared, const double* inv_freq, int B, int Hq, int Hk, int T,
                  int d, int rot_dim, int interleaved, float mscale, int dtype, void* stream) {
  return rope_any(q, k, q_out, k_out, strides, positions, positions_shared, inv_freq, B, Hq, Hk, T, d, rot_dim,
                  interleaved, mscale, dtype, 1.f, stream);
}

fa_status fa_rope_bwd(const void* dq_out, const void* dk_out, void* dq, void* dk, const long long* strides,
                      const int* positions, int positions_shared, const double* inv_freq, int B, int Hq, int Hk,
                      int T, int d, int rot_dim, int interleaved, float mscale, int dtype, void* stream) {
  return rope_any(dq_out, dk_out, dq, dk, strides, positions, positions_shared, inv_freq, B, Hq, Hk, T, d, rot_dim,
                  interleaved, mscale, dtype, -1.f, stream);
}

fa_status fa_rope_append_paged(const void* q, const void* k, const void* v, void* q_out, const long long* strides,
                               const int* positions, const int* slots, const double* inv_freq, void* k_pages,
                               void* v_pages, int B, int Hq, int Hkv, int T, int page_size, int num_pages, int d,
                               int rot_dim, int interleaved, float mscale, void* stream) {
  const fa_status st = check_rope(q, q_out, positions, inv_freq, B, Hq, Hkv, T, d, rot_dim, mscale, 2);
  if (st != FA_OK) return st;
  if (!strides || !k || !v || !slots || !k_pages || !v_pages || Hkv < 1 || num_pages < 1) return FA_ERR_INVALID_ARG;
  if (misaligned(k, 2) || misaligned(v, 2) || misaligned(slots, 4) || misaligned(k_pages, 16) ||
      misaligned(v_pages, 16))
    return FA_ERR_INVALID_ARG;
  if (page_size != 16 || static_cast<long long>(num_pages) * 16 >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const long long pool = 32ll * num_pages * Hkv * d;
  if (overlap(k_pages, pool, v_pages, pool)) return FA_ERR_INVALID_ARG;
  RopeParams p = {};
  p.q = side_of(q, q_out, strides, strides + 3, B, Hq, T);
  p.k = side_of(k, k_pages, strides + 6, nullptr, B, Hkv, T);
  p.v = side_of(v, v_pages, strides + 9, nullptr, B, Hkv, T);
  {
    // rows go to any slot while others are still read; q_out may be q and nothing else
    const long long bt4 = 4ll * B * T;
    const Rows out = rows_of(q_out, p.q.db, p.q.dh, p.q.dt, B, Hq, T, d, 2);
    if (outputs_meet(p.q, RopeSide{}, B, T, d, 2, positions, bt4, inv_freq, 4ll * rot_dim) ||
        rows_meet(out, rows_of(k, p.k.sb, p.k.sh, p.k.st, B, Hkv, T, d, 2)) ||
        rows_meet(out, rows_of(v, p.v.sb, p.v.sh, p.v.st, B, Hkv, T, d, 2)) || rows_meet(out, dense_rows(slots, bt4)))
      return FA_ERR_INVALID_ARG;
    for (const void* pages : {k_pages, v_pages}) {
      if (span_meets(q, p.q.sb, p.q.sh, p.q.st, B, Hq, T, d, 2, pages, pool) ||
          span_meets(q_out, p.q.db, p.q.dh, p.q.dt, B, Hq, T, d, 2, pages, pool) ||
          span_meets(k, p.k.sb, p.k.sh, p.k.st, B, Hkv, T, d, 2, pages, pool) ||
          span_meets(v, p.v.sb, p.v.sh, p.v.st, B, Hkv, T, d, 2, pages, pool) || overlap(positions, bt4, pages, pool) ||
          overlap(slots, bt4, pages, pool) || overlap(inv_freq, 4ll * rot_dim, pages, pool))
        return FA_ERR_INVALID_ARG;
    }
  }
  p.positions = positions;
  p.pos_sb = T;
  p.inv_freq = inv_freq;
  p.slots = slots;
  p.slot_stride = static_cast<long long>(Hkv) * d;
  p.num_slots = num_pages * 16;
  p.tokens = static_cast<long long>(B) * T;
  p.T = T;
  p.d = d;
  p.rot = rot_dim;
  p.mscale = mscale;
  p.sign = 1.f;
  p.err = device_error_word();
  if (!p.err) return static_cast<fa_status>(record_cuda_failure(cudaGetLastError()));
  return static_cast<fa_status>(launch_rope<__nv_bfloat16, true>(p, interleaved != 0, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
