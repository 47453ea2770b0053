// Attention of new tokens over the 4-bit cache: o = sum_j p_j v_j, p_j =
// exp(s_j - lse), s_j = scale q.k_j (capped), over the slots a token sees.
//
// The rows that read one key head (its group's q heads times the new tokens)
// are taken kRows at a time as the narrow side of m16n8k16 products:
//     S^T [16 keys, 8 rows] = K Q^T,     O^T [16 elements, 8 rows] += V^T P^T
// so the codes are always the 16-row operand, none of it padding.
//
// Codes as numbers.  A nibble c at bits 0-3 of a 16-bit half, read as fp16, is
// the subnormal c 2^-24, at bits 4-7 it is 16 c 2^-24; products with fp16
// numbers are exact in fp32.  So one AND makes a pair of operands, with no
// conversion, and q of odd elements carries the factor 1/16 (odd rows of O^T
// are divided at the end).  The offset 8 leaves K through the accumulators,
// which start at -8 2^-24 sum(q) of the group, and V by an exact fp16
// subtraction (a product with a constant operand instead would need
// accumulators for the sums of p s, registers that are not there).  Each
// group's scale multiplies S^T in fp32.
// Roundings: q is exact (bf16 into fp16 after a power of two that brings the
// row's largest magnitude to [2^14, 2^15); elements 2^-24 times smaller start
// to lose bits); a probability times its value scale is rounded to fp16.
//
// p s in fp16: 11 bits, where the outputs have 8; more would take two of every
// second product.  Every group of 32 channels has a base of its own, the exponent
// of the largest scale among a warp's first keys; raised by it, its scales are
// good while they lie in [2^-7, 2), 2^-5 to 2^3 of the base's own.  A row's
// reference R lies 2^10 below the largest score among keys whose scales are all
// good, and moves when that grows by more than 4 (log2 units); l = sum 2^(s_j - R)
// stays in fp32.  So the largest product of every group is in [2^3, 2^15), and the
// products below 2^-14, which lose up to 2^-25 each, together lose less than 2^-11
// of the sum over up to 2^17 keys of a warp.
// Other keys (of values 0, NaN, or much smaller or larger) take part in the same
// products but do not move R, unless a score of theirs is 2^24 above it: then, or
// where a product would leave fp16, or where a group of zeros gets its first
// values late, a step (from then on every step of the part, if R had to follow
// such a key) sorts its products into classes of 28 binades, a matrix product
// each, added up in fp32.
//
// Row tiles are of 8, the product's own width.  Tiles of 16 (two products on
// the same codes) halve the passes over the cache when a head has 9 or more
// rows, but double the registers of q and O: 41-45 us against 35 us for 16 rows
// a head (16 sequences, one head of 8192 keys), where the second pass comes out
// of the second-level cache.
//
// Work: all (sequence, head, row tile) pairs' key tiles of 128, and 3 more
// units for each pair, form one sequence, cut into equal runs, one per CTA;
// lengths are read on the device.  (A part costs a CTA about as much as 3 tiles,
// q's way in and the warps' sums: 16 sequences of unequal lengths, 75,000 keys
// on 8 heads, take 34 us with these units, 51 without.)
// A run's parts of pairs that other CTAs share go to the workspace as (R, l,
// O) records; a second kernel joins them in a fixed order and, if asked,
// turns the stored scores into probabilities and adds them to the weights.
// Short sequences (a capacity of up to 8 tiles) go a pair to a CTA instead, and
// nothing is joined: 128 heads of 512 slots take 13 us so and 19 split, 512 of
// 1024 32 and 35, 8 of 1024 14 and 12, 8 of 2048 would take 23 for 13.
//
// Four warps take 32 keys of a tile each, as two products side by side; the
// warps take turns in bringing tiles in by bulk copies through a ring of
// stages.  At three warps a scheduler what bounds it is the latency between
// their instructions (60% of the issue slots are taken, 53% of the ALU's).  Most
// of these are the ANDs, subtractions and packs around the products; the step
// therefore exists three times: for keys that every row sees (without predicates:
// 145 to 134 us below), for others, and class by class, in a loop of its own (in
// the others' loop it took registers: 149 us for 140).
// 64 sequences of 8191 keys on 8 heads, 32 q heads: 140 us, 605 MB at 4.3 TB/s
// (eight warps of 16 keys, one of them loading: 200 us); 144 if one group of all
// values is 0, 220 if every 64th value is, 330 class by class.  One sequence of
// 65,536 keys: 31 us, 75 MB; about 10 of them are the join, whose time is latency.
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kTileKeys = 128;
constexpr int kRows = 8;                   // rows of a row tile
constexpr int kWarps = 4;                  // 32 keys of a tile each, as two halves of 16
constexpr int kWholeTiles = 8;             // longest pair, in tiles, that one CTA takes alone
constexpr int kPartUnits = 3;              // cost of a part beside its tiles', in tiles
constexpr int kThreads = 32 * kWarps;
constexpr int kWeightKeys = 1024;          // keys of one head whose weights a CTA of the join adds to
// CTAs an SM, by registers (64 sequences of 8192 keys of 64: 94 us with four, 99 with three)
constexpr int ctas_per_sm(int D) { return D == 64 ? 4 : 3; }
constexpr float kRescale = 4.0f;
constexpr float kHead = 10.0f, kTail = 1.0f / 1024;  // a row's reference lies this far below the score that set it (log2 units)
constexpr float kAbove = 24.0f;            // how far above that a score of other keys may lie
// A group's scales are raised so that its base's lie in [2^-2, 2^-1); those good for products in one class are in
// [2^-7, 2): as bf16 exponent fields 01111xxx, these bits 0 and these 1, in pairs
constexpr uint32_t kBaseField = 125;
constexpr uint32_t kScaleZeros = 0xC000C000u, kScaleOnes = 0x3C003C00u;
constexpr uint32_t kNoBase = 0x7F00u;      // factor of a group whose scales have all been 0 so far: 2^127 leaves no other one small
constexpr float kTopProduct = 15.0f;       // products in one class stay below 2^15
constexpr int kClass = 28, kMidClass = 5;  // binades of a class; the class [2^-13, 2^15) among them
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Kv4FwdParams {
  bsa_kv4_cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int64_t qs[3], os[3];
  int32_t Hq, T, G, R;      // R = G * T rows per key head
  int32_t row_tiles;        // ceil(R / kRows)
  const int32_t *lens, *q_lens;
  float scale_log2;         // without a cap: scale * log2 e; with one: scale / cap
  float cap_log2;
  const float* sinks;
  int32_t n_sinks, sinks_kv;
  int32_t n_cta;
  int32_t whole;            // CTA c takes pair c, all of it
  float* rec_stat;          // [2 * n_cta][2][kRows]: R and l of a CTA's first and last part
  float* rec_o;             // [2 * n_cta][kRows][D]
  float* scores;            // [B * Hkv * row_tiles][capacity][score_stride], log2 units, or null
  int32_t score_stride;
  int32_t join_rows;        // blocks of the join kernel that merge rows ...
  int32_t rows_per_block;   // ... and how many of a pair's rows each takes (1, or all of a row tile)
  uint32_t* err;
  uint64_t wait_ns;
};

// ------------------------------------------------------------------ walk

// One (sequence, head, row tile) pair's place in the sequence of tiles.
struct Pair {
  int32_t b, len, nq;  // keys held; new tokens
  int32_t tiles;       // key tiles of each of the sequence's Hkv * row_tiles pairs ...
  int32_t units;       // ... and their cost: kPartUnits and one per tile, or 0
};

__device__ __forceinline__ Pair load_pair(const Kv4FwdParams& p, int32_t b, uint32_t* err) {
  Pair x;
  x.b = b;
  x.len = clamp_len(p.lens[b], p.c.capacity, err);
  x.nq = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
  x.tiles = x.nq > 0 ? (x.len + kTileKeys - 1) / kTileKeys : 0;
  x.units = x.tiles > 0 ? x.tiles + kPartUnits : 0;
  return x;
}

// Units of all sequences, and of the first ones up to b; every lane of the calling warp gets both.  Lengths outside
// the cache are reported to `err`, if there is one.
__device__ __forceinline__ int64_t total_units(const Kv4FwdParams& p, int32_t b, int64_t* before, uint32_t* err = nullptr) {
  const int lane = threadIdx.x & 31;
  const int64_t per = static_cast<int64_t>(p.c.Hkv) * p.row_tiles;
  int64_t sum = 0, head = 0;
  for (int32_t i = lane; i < p.c.B; i += 32) {
    const int64_t n = load_pair(p, i, err).units * per;
    sum += n;
    if (i < b) head += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    head += __shfl_xor_sync(0xffffffffu, head, o);
  }
  *before = head;
  return sum;
}

// CTAs that get a run of units (which may be short of a tile).  Of n, CTA c has
// units [c * total / n, (c + 1) * total / n); cta_of is the one that has unit t.
// A pair's first kPartUnits units are no tiles.
__device__ __forceinline__ int32_t runs(const Kv4FwdParams& p, int64_t total) {
  return static_cast<int32_t>(min(static_cast<int64_t>(p.n_cta), total));
}
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {  // of non-negative numbers, mostly small ones
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}
__device__ __forceinline__ int64_t first_unit(int64_t c, int64_t total, int32_t n) { return quotient(c * total, n); }
__device__ __forceinline__ int32_t cta_of(int64_t t, int64_t total, int32_t n) {
  return static_cast<int32_t>(quotient((t + 1) * n - 1, total));
}

// Cursor over a CTA's run: parts of pairs, each a range of key tiles.
struct Run {
  int64_t at, end;     // units of the run still to go
  int64_t seq0;        // first unit of sequence pair.b
  Pair pair;
  int32_t bh, rt;      // b * Hkv + h; row tile
  int32_t k0, k1;      // the part's key tiles
  bool whole;          // the part is the whole pair
  // places the cursor before unit `first` (warp-collective)
  __device__ __forceinline__ void init(const Kv4FwdParams& p, int64_t first, int64_t last) {
    at = first;
    end = last;
    const int lane = threadIdx.x & 31;
    const int64_t per = static_cast<int64_t>(p.c.Hkv) * p.row_tiles;
    seq0 = 0;
    int32_t b = 0;
    if (at < end) {
      for (int32_t b0 = 0;; b0 += 32) {
        const int64_t n = b0 + lane < p.c.B ? load_pair(p, b0 + lane, nullptr).units * per : 0;
        int64_t inc = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, seq0 + inc > at);
        if (past || b0 + 32 >= p.c.B) {
          const int l = past ? __ffs(past) - 1 : 31;
          b = b0 + l;
          seq0 += __shfl_sync(0xffffffffu, inc - n, l);
          break;
        }
        seq0 += __shfl_sync(0xffffffffu, inc, 31);
      }
      pair = load_pair(p, b, nullptr);
    }
  }
  // the whole of pair c (even one without tiles), as a run of one part
  __device__ __forceinline__ void init_whole(const Kv4FwdParams& p, int32_t c, uint32_t* err) {
    rt = c % p.row_tiles;
    bh = c / p.row_tiles;
    pair = load_pair(p, bh / p.c.Hkv, err);
    at = -1;
  }
  __device__ bool next(const Kv4FwdParams& p) {
    if (p.whole) {
      if (at == 0) return false;
      at = 0;
      k0 = 0;
      k1 = pair.tiles;
      whole = true;
      return true;
    }
    const int64_t per = static_cast<int64_t>(p.c.Hkv) * p.row_tiles;
    do {
      if (at >= end) return false;
      while (at >= seq0 + pair.units * per) {
        seq0 += pair.units * per;
        pair = load_pair(p, pair.b + 1, nullptr);
      }
      const int64_t i = at - seq0;
      const int32_t hr = static_cast<int32_t>(quotient(i, pair.units));
      bh = pair.b * p.c.Hkv + hr / p.row_tiles;
      rt = hr % p.row_tiles;
      const int32_t u0 = static_cast<int32_t>(i - static_cast<int64_t>(hr) * pair.units);
      const int32_t u1 = static_cast<int32_t>(min(static_cast<int64_t>(pair.units), u0 + (end - at)));
      at += u1 - u0;
      k0 = max(u0 - kPartUnits, 0);
      k1 = max(u1 - kPartUnits, 0);
    } while (k0 >= k1);
    whole = k0 == 0 && k1 == pair.tiles;
    return true;
  }
};

template <int D>
struct __align__(128) FwdShared {
  static constexpr int kStages = D == 128 ? 3 : 4;
  static constexpr int kAhead = kStages - 1;  // tiles issued before the one being computed
  static constexpr int kPad = D + 4;          // floats between rows of the merge buffer (bank spread)
  uint8_t k[kStages][kTileKeys * Kv4<D>::kRowBytes];
  uint8_t v[kStages][kTileKeys * Kv4<D>::kRowBytes];
  uint8_t ks[kStages][kTileKeys * Kv4<D>::kScaleBytes];
  uint8_t vs[kStages][kTileKeys * Kv4<D>::kScaleBytes];
  float merge[kWarps / 2][kRows * kPad];
  float stat[2][kWarps][kRows];
  float lse2[kRows];
  int32_t lim[kRows];
  uint64_t full[kStages], empty[kStages];
  Run ahead;            // the loader's place in the CTA's run
  int32_t ahead_tile;   // next key tile of that part
  uint32_t issued;      // tiles loaded, or on their way
  uint32_t abort_flag;
};

// ------------------------------------------------------------------ products

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same into fresh accumulators that start at z0 (even column) and z1.
__device__ __forceinline__ void mma_f16_from(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1, float z0, float z1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(z0), "f"(z1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two fp16 numbers minus a constant (subnormals all: exact).
__device__ __forceinline__ uint32_t minus8(uint32_t x, uint32_t c) {
  uint32_t y;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(c));
  return y;
}

// Two bf16 numbers times a power of two (exact).
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}

template <int N>
__device__ __forceinline__ void lds(uint32_t (&w)[N], const void* p) {
  if constexpr (N == 4) {
    const uint4 x = *static_cast<const uint4*>(p);
    w[0] = x.x;
    w[1] = x.y;
    w[2] = x.z;
    w[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *static_cast<const uint2*>(p);
    w[0] = x.x;
    w[1] = x.y;
  } else {
    w[0] = *static_cast<const uint32_t*>(p);
  }
}

// Finite magnitudes of two bf16 numbers (0 for a NaN or an infinity).
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  const uint32_t lo = w & 0x7FFFu, hi = w & 0x7FFF0000u;
  return (lo < 0x7F80u ? lo : 0u) | (hi < 0x7F800000u ? hi : 0u);
}

// What raises the scales of a group whose first keys' largest is `top` (bf16 bits, not 0): a power of two, as bf16 bits.
__device__ __forceinline__ uint32_t raising_bits(uint32_t top) {
  return min(127u + kBaseField - (top >> 7), 253u) << 7;
}
// One over that.
__device__ __forceinline__ float lowering(uint32_t bits) {
  const uint32_t e = 254u - (bits >> 7);
  return __uint_as_float(e ? e << 23 : 0x00400000u);
}

// Exponent of the power of two above a key's scales.
template <int W>
__device__ __forceinline__ float exponent_above(const uint32_t (&w)[W]) {
  uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < W; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return static_cast<float>(static_cast<int>(max(m & 0xFFFFu, m >> 16) >> 7) - 126);
}

// Class of a product, 1 to 9, 0 for one too small to count; a NaN or an infinity counts to the middle one.
__device__ __forceinline__ int class_of(float w) {
  const uint32_t e = (__float_as_uint(w) >> 23) & 255u;  // (the middle one: 114 to 141)
  return e == 255u ? kMidClass : min(static_cast<int>((e + 26u) / kClass), 9);
}

// ------------------------------------------------------------------ results

// Adds a row's sinks: (R, l) -> its logsumexp in log2 units and the factor of
// the unnormalised output.
__device__ __forceinline__ float finish_row(const Kv4FwdParams& p, int32_t h, float R, float l, float& factor) {
  float lse2 = l == 0.f ? -INFINITY : R + log2f(l);
  factor = l == 0.f ? 0.f : 1.f / l;
  if (p.n_sinks > 0) {
    const float* z = p.sinks + (p.sinks_kv ? h * p.n_sinks : 0);
    float m = lse2;
    for (int j = 0; j < p.n_sinks; ++j) m = fmaxf(m, z[j] * kLog2e);
    float tot = lse2 == -INFINITY ? 0.f : ex2_approx(lse2 - m);
    for (int j = 0; j < p.n_sinks; ++j) tot += ex2_approx(fmaf(z[j], kLog2e, -m));
    const float all = m == -INFINITY ? -INFINITY : m + log2f(tot);
    if (l != 0.f) factor *= ex2_approx(lse2 - all);
    lse2 = all;
  }
  return lse2;
}

// Row r (q head r / T of the group, token r % T) of pair bh.
__device__ __forceinline__ int64_t lse_index(const Kv4FwdParams& p, int32_t bh, int32_t r) {
  const int32_t b = bh / p.c.Hkv, hq = bh % p.c.Hkv * p.G + r / p.T;
  return (static_cast<int64_t>(b) * p.Hq + hq) * p.T + r % p.T;
}
__device__ __forceinline__ __nv_bfloat16* o_row(const Kv4FwdParams& p, int32_t bh, int32_t r) {
  const int32_t b = bh / p.c.Hkv, hq = bh % p.c.Hkv * p.G + r / p.T;
  return p.o + b * p.os[0] + hq * p.os[1] + (r % p.T) * p.os[2];
}

__device__ __forceinline__ void store_o4(__nv_bfloat16* o, const float4& x, float f) {
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(x.x * f, x.y * f), pack_bf16x2(x.z * f, x.w * f));
}

// Slots that row r of a pair sees: the first `row_limit` ones.
__device__ __forceinline__ int32_t row_limit(const Kv4FwdParams& p, const Pair& pair, int32_t r) {
  const int32_t t = r % p.T;
  return r < p.R && t < pair.nq ? max(0, pair.len - pair.nq + t + 1) : 0;
}

// The scores of keys j0 + i * step over the rows of a row tile (of pair `head`), and their probabilities, of the rows
// that see the key, added to w[i].
template <int N>
struct KeyScores {
  float2 v[N][kRows / 2];
  __device__ __forceinline__ void load(const Kv4FwdParams& p, int64_t head, int32_t j0, int32_t step, int32_t len) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t j = j0 + i * step;
      const float2* sc = reinterpret_cast<const float2*>(p.scores + (head * p.c.capacity + j) * p.score_stride);
#pragma unroll
      for (int r = 0; r < kRows / 2; ++r) v[i][r] = j < len && 2 * r < p.score_stride ? sc[r] : make_float2(0.f, 0.f);
    }
  }
  __device__ __forceinline__ void add(int32_t j0, int32_t step, const float* lse2, const int32_t* lim, float* w) const {
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float l = lse2[r];
      const int32_t n = lim[r];
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (j0 + i * step < n) w[i] += ex2_approx((r & 1 ? v[i][r / 2].y : v[i][r / 2].x) - l);
    }
  }
};

template <int D, bool kCap>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D)) kv4_fwd_kernel(const __grid_constant__ Kv4FwdParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Sh = FwdShared<D>;
  Sh& s = *reinterpret_cast<Sh*>(smem_raw);
  constexpr int kStages = Sh::kStages, kGroups = Kv4<D>::kGroups;
  constexpr int kRowBytes = Kv4<D>::kRowBytes, kScaleBytes = Kv4<D>::kScaleBytes;
  const int warp = warp_id(), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kWarps);
    }
    fence_mbar_init();
  }
  __syncthreads();
  // (not before a join: its early blocks would wait in the place of CTAs of the call after next, which
  // took 16 sequences of 8192 keys with 16 rows a head from 38 to 54 us a call)
  if (p.whole) griddep_launch_dependents();
  griddep_wait();
  const WaitCtl wc{p.err, &s.abort_flag, p.wait_ns};
  Run run;
  if (p.whole) {
    run.init_whole(p, blockIdx.x, threadIdx.x == 0 ? p.err : nullptr);
  } else {
    int64_t none;
    // (every CTA goes through all sequences; the first one's first warp reports)
    const int64_t total = total_units(p, 0, &none, blockIdx.x == 0 && warp == 0 ? p.err : nullptr);
    const int32_t n_cta = runs(p, total);
    if (static_cast<int32_t>(blockIdx.x) >= n_cta) return;
    run.init(p, first_unit(blockIdx.x, total, n_cta), first_unit(blockIdx.x + 1, total, n_cta));
  }

  // One lane: tile `n` of the run into its stage, if there is one; true if that went well.
  auto load_tile = [&](uint32_t n) -> bool {
    const uint32_t st = n % kStages;
    // (also orders this loader after the one before it, which another warp may have been)
    if (n >= static_cast<uint32_t>(kStages) && !mbar_wait(&s.empty[st], (n / kStages - 1) & 1u, wc)) return false;
    if (s.ahead_tile >= s.ahead.k1) {
      do {
        if (!s.ahead.next(p)) return true;
      } while (s.ahead.k0 >= s.ahead.k1);
      s.ahead_tile = s.ahead.k0;
    }
    const int32_t kt = s.ahead_tile++;
    const int64_t key = static_cast<int64_t>(s.ahead.bh) * p.c.capacity + static_cast<int64_t>(kt) * kTileKeys;
    // whole sixteens of keys: the capacity is a multiple of 16
    const uint32_t keys = static_cast<uint32_t>((min(s.ahead.pair.len - kt * kTileKeys, kTileKeys) + 15) & ~15);
    mbar_arrive_expect_tx(&s.full[st], keys * 2 * (kRowBytes + kScaleBytes));
    bulk_load(s.k[st], static_cast<const uint8_t*>(p.c.k_codes) + key * kRowBytes, keys * kRowBytes, &s.full[st]);
    bulk_load(s.ks[st], static_cast<const uint8_t*>(p.c.k_scales) + key * kScaleBytes, keys * kScaleBytes, &s.full[st]);
    bulk_load(s.v[st], static_cast<const uint8_t*>(p.c.v_codes) + key * kRowBytes, keys * kRowBytes, &s.full[st]);
    bulk_load(s.vs[st], static_cast<const uint8_t*>(p.c.v_scales) + key * kScaleBytes, keys * kScaleBytes, &s.full[st]);
    s.issued = n + 1;
    return true;
  };
  bool ok = true;
  if (threadIdx.x == 0) {
    s.ahead = run;
    s.ahead.k1 = 0;
    s.ahead_tile = 0;
    s.issued = 0;
    for (int i = 0; ok && i < Sh::kAhead; ++i) ok = load_tile(i);
  }
  ok = __syncthreads_and(ok);

  const int g8 = lane >> 2, t4 = lane & 3;  // fragment row / column pair
  // V rows of this lane: keys 2 t4, 2 t4 + 1 (+ 8), the one that lies in the
  // other bank half first in lanes 2 and 3 (kv4.cuh), put right by the byte selectors
  const int v_first = t4 >> 1;
  const uint32_t sel_lo = v_first ? 0x1054u : 0x5410u, sel_hi = v_first ? 0x3276u : 0x7632u;
  // this lane's places in a stage
  const int k_at = (warp * 32 + g8) * kRowBytes + t4 * (kRowBytes / 4), s_at = (warp * 32 + g8) * kScaleBytes;
  const int v_at = (warp * 32 + 2 * t4 + v_first) * kRowBytes + (D == 128 ? g8 ^ ((t4 & 1) << 2) : g8) * (kRowBytes / 8);
  const int v_next = v_first ? -kRowBytes : kRowBytes;
  uint32_t n = 0, st = 0, parity = 0;
  bool first_part = true;
  while (run.next(p)) {
    const int32_t h = run.bh % p.c.Hkv;
    const int64_t head = static_cast<int64_t>(run.bh) * p.row_tiles + run.rt;
    // Q as fp16 operands, the start of K's accumulators, and per column its factor and last slot
    uint32_t qb[kGroups][4];
    float init[kGroups][2], qf[2];
    int32_t lim[2];
    int32_t lim_min = INT32_MAX, lim_max = 0;
    const int32_t r = run.rt * kRows + g8;  // this lane's row while loading Q
    const bool in = r < p.R;
    const int32_t t = in ? r % p.T : 0;
    uint4 raw[kGroups];
    uint32_t mx = 0;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      raw[g] = in ? *reinterpret_cast<const uint4*>(p.q + run.pair.b * p.qs[0] + (h * p.G + r / p.T) * p.qs[1] + t * p.qs[2] +
                                                    32 * g + 8 * t4)
                  : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) mx = max(mx, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    }
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // power of two that brings the row's largest magnitude to [2^14, 2^15)
    const int e = mx == 0 || mx >= 0x7F80u ? 0 : 14 + 127 - static_cast<int>(max(mx >> 7, 1u));
    const float up = exp2f(static_cast<float>(e / 2)), up2 = exp2f(static_cast<float>(e - e / 2));
    float sum[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]) * up * up2;
        x[2 * i + 1] = bf16_hi(w[i]) * up * up2 * 0.0625f;
      }
      sum[g] = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {  // elements 2 hf (+4) and 2 hf + 1 (+4): see kv4.cuh
        const __half2 even = __floats2half2_rn(x[2 * hf], x[2 * hf + 4]);
        const __half2 odd = __floats2half2_rn(x[2 * hf + 1], x[2 * hf + 5]);
        qb[g][2 * hf] = *reinterpret_cast<const uint32_t*>(&even);
        qb[g][2 * hf + 1] = *reinterpret_cast<const uint32_t*>(&odd);
        const float2 fe = __half22float2(even), fo = __half22float2(odd);
        sum[g] += fe.x + fe.y + 16.f * (fo.x + fo.y);
      }
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 1);
      sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], 2);
    }
    const float f = p.scale_log2 * 16777216.f * exp2f(static_cast<float>(-e));
    const int32_t last = in && t < run.pair.nq ? max(0, run.pair.len - run.pair.nq + t + 1) : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // this lane's columns are rows 2 t4 and 2 t4 + 1
      const int from = 4 * (2 * t4 + i);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) init[g][i] = __shfl_sync(0xffffffffu, sum[g], from) * (-8.f / 16777216.f);
      qf[i] = __shfl_sync(0xffffffffu, f, from);
      lim[i] = __shfl_sync(0xffffffffu, last, from);
    }
    int32_t lo = in ? last : INT32_MAX, hi = last;
#pragma unroll
    for (int o = 4; o < 32; o *= 2) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lim_min = min(lim_min, lo);
    lim_max = max(lim_max, hi);

    float acc[2 * kGroups][4];
    float R[2], l[2];
#pragma unroll
    for (int j = 0; j < 2 * kGroups; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    R[0] = R[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    // (uniform over the warp) the factor of each group's scales; is there a group without a base; has there been a
    // step; are all products to be taken class by class from here on
    uint32_t down[kGroups / 2];
#pragma unroll
    for (int i = 0; i < kGroups / 2; ++i) down[i] = kNoBase * 0x00010001u;
    bool open = true, begun = false, careful = false;
    // bits that a good pair of raised scales has none of, and all of (groups without a base: only zeros are good)
    struct Good {
      uint32_t zeros, ones;
    };
    auto good = [&](int i) __attribute__((always_inline)) -> Good {
      Good x{kScaleZeros, kScaleOnes};
      if (open) {
        const uint32_t none = ((down[i] & 0xFFFFu) == kNoBase ? 0xFFFFu : 0u) | ((down[i] >> 16) == kNoBase ? 0xFFFF0000u : 0u);
        x.zeros |= none;
        x.ones &= ~none;
      }
      return x;
    };
    // before a step while there are groups without a base: bases for those that get values now
    auto look = [&](int key0) __attribute__((always_inline)) {
      open = false;
#pragma unroll
      for (int i = 0; i < kGroups / 2; ++i) {
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (key0 + 8 * u + g8 < run.pair.len)
            top = __vmaxu2(top, finite_bits(*reinterpret_cast<const uint32_t*>(s.vs[st] + s_at + u * 8 * kScaleBytes + 4 * i)));
#pragma unroll
        for (int o = 4; o < 32; o *= 2) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int sh = 0; sh < 32; sh += 16) {
          if (((down[i] >> sh) & 0xFFFFu) != kNoBase) continue;
          const uint32_t t = (top >> sh) & 0xFFFFu;
          if (t) {
            down[i] = (down[i] & ~(0xFFFFu << sh)) | raising_bits(t) << sh;
            careful |= begun;  // (the probabilities so far may be far above this group's first)
          } else {
            open = true;
          }
        }
      }
      begun = true;
    };
    // 32 keys; kAll: every row sees all of them; kOne: products of one class (false, and nothing done, if they are not)
    auto step = [&](auto all, auto one, int key0) __attribute__((always_inline)) -> bool {
      constexpr bool kAll = decltype(all)::value, kOne = decltype(one)::value;
      // ---- scores of both halves
      float x[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t ka[kGroups], kb[kGroups], sa[kGroups / 2], sb[kGroups / 2];
        lds(ka, s.k[st] + k_at + u * 16 * kRowBytes);
        lds(kb, s.k[st] + k_at + (u * 16 + 8) * kRowBytes);
        lds(sa, s.ks[st] + s_at + u * 16 * kScaleBytes);
        lds(sb, s.ks[st] + s_at + (u * 16 + 8) * kScaleBytes);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float fa = g & 1 ? bf16_hi(sa[g / 2]) : bf16_lo(sa[g / 2]);
          const float fb = g & 1 ? bf16_hi(sb[g / 2]) : bf16_lo(sb[g / 2]);
          const uint32_t a8 = ka[g] >> 8, b8 = kb[g] >> 8;
          float c[4];
          mma_f16_from(c, ka[g] & 0x000F000Fu, kb[g] & 0x000F000Fu, ka[g] & 0x00F000F0u, kb[g] & 0x00F000F0u,
                       qb[g][0], qb[g][1], init[g][0], init[g][1]);
          mma_f16(c, a8 & 0x000F000Fu, b8 & 0x000F000Fu, a8 & 0x00F000F0u, b8 & 0x00F000F0u, qb[g][2], qb[g][3]);
          x[u][0] = g ? fmaf(fa, c[0], x[u][0]) : fa * c[0];
          x[u][1] = g ? fmaf(fa, c[1], x[u][1]) : fa * c[1];
          x[u][2] = g ? fmaf(fb, c[2], x[u][2]) : fb * c[2];
          x[u][3] = g ? fmaf(fb, c[3], x[u][3]) : fb * c[3];
        }
      }
      // ---- value scales, raised
      uint32_t va[2][kGroups / 2], vb[2][kGroups / 2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        lds(va[u], s.vs[st] + s_at + u * 16 * kScaleBytes);
        lds(vb[u], s.vs[st] + s_at + (u * 16 + 8) * kScaleBytes);
      }
      uint32_t bad_a[2] = {}, bad_b[2] = {}, bad = 0;
#pragma unroll
      for (int i = 0; i < kGroups / 2; ++i) {
        const Good y = good(i);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          va[u][i] = mul_bf16x2(va[u][i], down[i]);
          vb[u][i] = mul_bf16x2(vb[u][i], down[i]);
          if constexpr (!kAll) {  // (whatever slots past the length hold changes nothing)
            if (key0 + 16 * u + g8 >= run.pair.len) va[u][i] = y.ones;
            if (key0 + 16 * u + g8 + 8 >= run.pair.len) vb[u][i] = y.ones;
          }
          if constexpr (!kAll) {
            bad_a[u] |= (va[u][i] & y.zeros) | (~va[u][i] & y.ones);
            bad_b[u] |= (vb[u][i] & y.zeros) | (~vb[u][i] & y.ones);
          }
        }
        bad |= ((va[0][i] | vb[0][i] | va[1][i] | vb[1][i]) & y.zeros) | (~(va[0][i] & vb[0][i] & va[1][i] & vb[1][i]) & y.ones);
      }
      const bool odd = __any_sync(0xffffffffu, bad);
      if (odd && kOne && (kAll || open)) return false;
      // ---- softmax
      float pr[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[u][i] *= qf[i & 1];
          if constexpr (kCap) x[u][i] = p.cap_log2 * tanh_nan(x[u][i]);
        }
      if constexpr (!kAll) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 16 * u + g8 + (i >> 1) * 8 >= lim[i & 1]) x[u][i] = -INFINITY;
      }
      if (p.scores && 2 * t4 < p.score_stride) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (key0 + 16 * u >= p.c.capacity) continue;
          float* out = p.scores + (head * p.c.capacity + key0 + 16 * u + g8) * p.score_stride + 2 * t4;
          *reinterpret_cast<float2*>(out) = make_float2(x[u][0], x[u][1]);
          *reinterpret_cast<float2*>(out + 8 * p.score_stride) = make_float2(x[u][2], x[u][3]);
        }
      }
      float m[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) m[i] = fmaxf(fmaxf(x[0][i], x[0][i + 2]), fmaxf(x[1][i], x[1][i + 2]));
      auto over_keys = [&](float(&y)[2]) __attribute__((always_inline)) {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) {
          y[0] = fmaxf(y[0], __shfl_xor_sync(0xffffffffu, y[0], o));
          y[1] = fmaxf(y[1], __shfl_xor_sync(0xffffffffu, y[1], o));
        }
      };
      over_keys(m);
      if (!kAll && odd) {
        // the reference follows the keys all of whose scales are good, unless another is far above it
        float near[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!bad_a[u]) near[i] = fmaxf(near[i], x[u][i]);
            if (!bad_b[u]) near[i] = fmaxf(near[i], x[u][i + 2]);
          }
        over_keys(near);
        bool far = m[0] > fmaxf(near[0], R[0] + kHead) + kAbove || m[1] > fmaxf(near[1], R[1] + kHead) + kAbove;
        if constexpr (kOne) {  // nor may a product leave fp16
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float top = (near[i] > R[i] + (kHead + kRescale) ? near[i] - kHead : R[i]) + kTopProduct;
#pragma unroll
            for (int u = 0; u < 2; ++u)
              far |= x[u][i] + exponent_above(va[u]) > top || x[u][i + 2] + exponent_above(vb[u]) > top;
          }
        }
        if (__any_sync(0xffffffffu, far)) {
          if constexpr (kOne) return false;
          careful = true;
        } else {
          m[0] = near[0];
          m[1] = near[1];
        }
      }
      if (__any_sync(0xffffffffu, m[0] > R[0] + (kHead + kRescale) || m[1] > R[1] + (kHead + kRescale))) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (uniform over the lanes of a column)
          const float to = m[i] > R[i] + (kHead + kRescale) ? m[i] - kHead : R[i];
          const float f = R[i] == -INFINITY ? 0.f : ex2_approx(R[i] - to);
          R[i] = to;
          l[i] *= f;
#pragma unroll
          for (int j = 0; j < 2 * kGroups; ++j) {
            acc[j][i] *= f;
            acc[j][i + 2] *= f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ref = R[i] == -INFINITY ? 0.f : R[i];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          pr[u][i] = ex2_approx(x[u][i] - ref);
          pr[u][i + 2] = ex2_approx(x[u][i + 2] - ref);
        }
        l[i] += (pr[0][i] + pr[0][i + 2]) + (pr[1][i] + pr[1][i + 2]);
      }
      // ---- output, a half at a time
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t v0[kGroups / 2], v1[kGroups / 2], v8[kGroups / 2], v9[kGroups / 2];
        const uint8_t* vrow = s.v[st] + v_at + u * 16 * kRowBytes;
        lds(v0, vrow);
        lds(v1, vrow + v_next);
        lds(v8, vrow + 8 * kRowBytes);
        lds(v9, vrow + 8 * kRowBytes + v_next);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          // probabilities times value scales, transposed into the second product's operand
          const float fa = g & 1 ? bf16_hi(va[u][g / 2]) : bf16_lo(va[u][g / 2]);
          const float fb = g & 1 ? bf16_hi(vb[u][g / 2]) : bf16_lo(vb[u][g / 2]);
          float w[4] = {pr[u][0] * fa, pr[u][1] * fa, pr[u][2] * fb, pr[u][3] * fb};
          if constexpr (!kAll) {  // (an unseen slot's scale may be anything)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (x[u][i] == -INFINITY) w[i] = 0.f;
          }
          const uint32_t sel = g & 1 ? sel_hi : sel_lo;
          const uint32_t lo = __byte_perm(v0[g / 2], v1[g / 2], sel), hi = __byte_perm(v8[g / 2], v9[g / 2], sel);
          // elements 4 g8 + 0..3 of the group: rows g8 and (times 16) g8 + 8 of two products
          const uint32_t a0 = minus8(lo & 0x000F000Fu, 0x00080008u), a1 = minus8(lo & 0x00F000F0u, 0x00800080u);
          const uint32_t a2 = minus8(hi & 0x000F000Fu, 0x00080008u), a3 = minus8(hi & 0x00F000F0u, 0x00800080u);
          const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
          const uint32_t c0 = minus8(lo8 & 0x000F000Fu, 0x00080008u), c1 = minus8(lo8 & 0x00F000F0u, 0x00800080u);
          const uint32_t c2 = minus8(hi8 & 0x000F000Fu, 0x00080008u), c3 = minus8(hi8 & 0x00F000F0u, 0x00800080u);
          if constexpr (kOne) {
            const uint32_t b0 = transpose8x8(pack_f16x2(w[0], w[1])), b1 = transpose8x8(pack_f16x2(w[2], w[3]));
            mma_f16(acc[2 * g], a0, a1, a2, a3, b0, b1);
            mma_f16(acc[2 * g + 1], c0, c1, c2, c3, b0, b1);
          } else {
            int cls[4];
            uint32_t have = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              cls[i] = class_of(w[i]);
              have |= 1u << cls[i];
            }
            have = __reduce_or_sync(0xffffffffu, have) & ~1u;
            while (have) {
              const int c = __ffs(have) - 1;
              have &= have - 1;
              const float into = __uint_as_float(static_cast<uint32_t>(127 + kClass * (kMidClass - c)) << 23);
              const float back = __uint_as_float(static_cast<uint32_t>(127 - kClass * (kMidClass - c)) << 23);
              float y[4], x0[4] = {}, x1[4] = {};
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = cls[i] == c ? w[i] * into : 0.f;
              const uint32_t b0 = transpose8x8(pack_f16x2(y[0], y[1])), b1 = transpose8x8(pack_f16x2(y[2], y[3]));
              mma_f16(x0, a0, a1, a2, a3, b0, b1);
              mma_f16(x1, c0, c1, c2, c3, b0, b1);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                acc[2 * g][i] = fmaf(x0[i], back, acc[2 * g][i]);
                acc[2 * g + 1][i] = fmaf(x1[i], back, acc[2 * g + 1][i]);
              }
            }
          }
        }
      }
      return true;
    };

    int32_t kt = run.k0;
    auto tiles = [&](auto one) __attribute__((always_inline)) {
      constexpr bool kOne = decltype(one)::value;
      for (; kt < run.k1; ++kt, ++n) {
        // (after a wait that ran out the loop goes on without waiting, on whatever
        // the stages hold: the barriers between the warps stay matched)
        if (ok) ok = mbar_wait_warp(&s.full[st], parity, wc);
        const int32_t key0 = kt * kTileKeys + warp * 32;
        if (key0 < lim_max) {
          if constexpr (kOne) {
            const bool all = __all_sync(0xffffffffu, key0 + 32 <= lim_min);
            if (!begun) look(key0);
            if (careful || (!(all && step(std::true_type{}, one, key0)) && !step(std::false_type{}, one, key0))) return;
          } else {
            if (open) look(key0);
            step(std::false_type{}, one, key0);
          }
        }
        // (at the end: the stage it goes to, the last tile's, is long released; before this warp's own release, which
        // hands the loader's place on to the next warp)
        if (static_cast<int>(n % kWarps) == warp) {
          if (lane == 0 && ok) ok = load_tile(n + Sh::kAhead);
          ok = __all_sync(0xffffffffu, ok);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[st]);
        if (++st == kStages) {
          st = 0;
          parity ^= 1u;
        }
        if (!kOne && !careful) {
          ++kt;
          ++n;
          return;
        }
      }
    };
    while (kt < run.k1) {
      tiles(std::true_type{});
      tiles(std::false_type{});  // (the tile that is not of one class)
    }

    // ---- the warps' parts into one
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      if (g8 == 0) {
        s.stat[0][warp][2 * t4 + i] = R[i] + kHead;  // (sums as if for the score that set the reference)
        s.stat[1][warp][2 * t4 + i] = l[i] * kTail;
      }
    }
    __syncthreads();
    auto slot = [&](int i, int g) -> float4* {
      return reinterpret_cast<float4*>(&s.merge[warp % (kWarps / 2)][(2 * t4 + i) * Sh::kPad + 32 * g + 4 * g8]);
    };
    // this warp's share of a column's output, for the common reference
    auto share = [&](int i, int g) -> float4 {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s.stat[0][w][2 * t4 + i]);
      const float f = R[i] == -INFINITY ? (l[i] == 0.f ? 0.f : 1.f) : ex2_approx(R[i] + kHead - m);
      const float even = f * (kTail * 16777216.f), odd = even * 0.0625f;
      // (by itself: it may be far from 1)
      const float up_back = lowering((down[g / 2] >> (g & 1) * 16) & 0xFFFFu);
      return make_float4(acc[2 * g][i] * even * up_back, acc[2 * g][i + 2] * odd * up_back,
                         acc[2 * g + 1][i] * even * up_back, acc[2 * g + 1][i + 2] * odd * up_back);
    };
    if (warp >= kWarps / 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) *slot(i, g) = share(i, g);
    }
    __syncthreads();
    if (warp < kWarps / 2) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          float4* at = slot(i, g);
          const float4 a = *at, b = share(i, g);
          *at = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
        }
    }
    __syncthreads();
    const int32_t rec = 2 * static_cast<int32_t>(blockIdx.x) + (first_part ? 0 : 1);
    for (int idx = threadIdx.x; idx < kRows * D / 4; idx += kThreads) {
      const int row = idx / (D / 4), d = idx % (D / 4) * 4;
      float m = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s.stat[0][w][row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (s.stat[1][w][row] != 0.f) L += s.stat[1][w][row] * (m == -INFINITY ? 1.f : ex2_approx(s.stat[0][w][row] - m));
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps / 2; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(&s.merge[w][row * Sh::kPad + d]);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      if (run.whole) {
        const int32_t r = run.rt * kRows + row;
        if (r < p.R) {
          float f;
          const float lse2 = finish_row(p, h, m, L, f);
          store_o4(o_row(p, run.bh, r) + d, x, f);
          if (d == 0) {
            s.lse2[row] = lse2;
            p.lse[lse_index(p, run.bh, r)] = lse2 * kLn2;
          }
        }
      } else {
        *reinterpret_cast<float4*>(p.rec_o + (static_cast<int64_t>(rec) * kRows + row) * D + d) = x;
        if (d == 0) {
          p.rec_stat[rec * 2 * kRows + row] = m;
          p.rec_stat[rec * 2 * kRows + kRows + row] = L;
        }
      }
    }
    first_part = false;
    if (p.whole && p.scores) {
      // (one row tile) this CTA's own scores into probabilities
      if (threadIdx.x < kRows) s.lim[threadIdx.x] = row_limit(p, run.pair, static_cast<int32_t>(threadIdx.x));
      __syncthreads();
      for (int32_t j = threadIdx.x; j < run.pair.len; j += kThreads) {
        float w[1] = {};
        KeyScores<1> x;
        x.load(p, run.bh, j, 0, run.pair.len);
        x.add(j, 0, s.lse2, s.lim, w);
        p.c.weights[static_cast<int64_t>(run.bh) * p.c.capacity + j] += w[0];
      }
    }
    __syncthreads();  // the next part, maybe of few tiles, writes `stat` and `merge` again
  }
  if (!__syncthreads_and(ok) && threadIdx.x == 0) {
    // the copies in flight land before the CTA exits
    uint32_t dummy_abort = 0;
    WaitCtl dw{nullptr, &dummy_abort, p.wait_ns};
    for (uint32_t i = s.issued > kStages ? s.issued - kStages : 0; i < s.issued; ++i)
      (void)mbar_wait(&s.full[i % kStages], (i / kStages) & 1u, dw);
  }
}

// The records of a pair: CTAs c0 .. c1, a CTA's being its first part unless its
// run began in an earlier pair (which only c0's can have).
struct Records {
  int32_t c0, c1, first;  // first: c0's record
  int32_t tiles;
  __device__ __forceinline__ int32_t of(int32_t c) const { return c == c0 ? first : 2 * c; }
};

__device__ __forceinline__ Records pair_records(const Kv4FwdParams& p, int32_t bh, int32_t rt, const Pair& pair) {
  const int32_t b = bh / p.c.Hkv, h = bh % p.c.Hkv;
  int64_t before;
  const int64_t total = total_units(p, b, &before);
  Records x{0, 0, 0, pair.tiles};
  if (pair.tiles > 0) {
    const int32_t n = runs(p, total);
    const int64_t begin = before + (static_cast<int64_t>(h) * p.row_tiles + rt) * pair.units;
    x.c0 = cta_of(begin + kPartUnits, total, n);
    x.c1 = cta_of(begin + pair.units - 1, total, n);
    x.first = 2 * x.c0 + (first_unit(x.c0, total, n) < begin ? 1 : 0);
  }
  return x;
}

constexpr int kJoinThreads = 256;

// Joins records: every row of the pair's reference and sum, by the whole CTA.
__device__ __forceinline__ void join_stats(const Kv4FwdParams& p, const Records& x, float (*part)[2][kRows], float* R, float* L) {
  constexpr int kSub = 32 / kRows;  // records side by side in a warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane % kRows;
  float m = -INFINITY, l = 0.f;
  for (int32_t c = x.c0 + warp * kSub + lane / kRows; c <= x.c1; c += kJoinThreads / kRows) {
    const float* st = p.rec_stat + x.of(c) * 2 * kRows + row;
    const float mc = st[0], lc = st[kRows];
    const float to = fmaxf(m, mc);
    l = (l == 0.f ? 0.f : l * (to == -INFINITY ? 1.f : ex2_approx(m - to))) +
        (lc == 0.f ? 0.f : lc * (to == -INFINITY ? 1.f : ex2_approx(mc - to)));
    m = to;
  }
  auto add = [](float& m, float& l, float mc, float lc) {
    const float to = fmaxf(m, mc);
    l = (l == 0.f ? 0.f : l * (to == -INFINITY ? 1.f : ex2_approx(m - to))) +
        (lc == 0.f ? 0.f : lc * (to == -INFINITY ? 1.f : ex2_approx(mc - to)));
    m = to;
  };
#pragma unroll
  for (int o = kRows; o < 32; o *= 2) {
    const float mc = __shfl_xor_sync(0xffffffffu, m, o), lc = __shfl_xor_sync(0xffffffffu, l, o);
    add(m, l, mc, lc);
  }
  __syncthreads();
  if (lane < kRows) {
    part[warp][0][row] = m;
    part[warp][1][row] = l;
  }
  __syncthreads();
  if (threadIdx.x < kRows) {
    m = part[0][0][threadIdx.x];
    l = part[0][1][threadIdx.x];
    for (int w = 1; w < kJoinThreads / 32; ++w) add(m, l, part[w][0][threadIdx.x], part[w][1][threadIdx.x]);
    R[threadIdx.x] = m;
    L[threadIdx.x] = l;
  }
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const __grid_constant__ Kv4FwdParams p) {
  constexpr int kVec = D / 4;                 // lanes (float4) of one row
  constexpr int kSplit = kJoinThreads / kVec;  // records read side by side
  __shared__ float4 part[kSplit][kVec];
  __shared__ float stats[kJoinThreads / 32][2][kRows], R[kRows], L[kRows];
  griddep_wait();
  if (static_cast<int32_t>(blockIdx.x) < p.join_rows) {
    // ---- output of one row, or of all rows of a pair side by side
    const int32_t blocks = p.rows_per_block == 1 ? min(p.R, kRows) : 1;  // per pair (a last, shorter row tile has idle ones)
    const int32_t hr = static_cast<int32_t>(blockIdx.x) / blocks, rt = hr % p.row_tiles, bh = hr / p.row_tiles;
    const Records x = pair_records(p, bh, rt, load_pair(p, bh / p.c.Hkv, nullptr));
    if (x.tiles > 0 && x.c0 == x.c1) return;  // one CTA had all of it
    const int lane = threadIdx.x % kVec, sub = threadIdx.x / kVec;
    const int split = kSplit / p.rows_per_block;  // records of a row read side by side
    const int row = p.rows_per_block == 1 ? static_cast<int32_t>(blockIdx.x) % blocks : sub / split;
    const int32_t r = rt * kRows + row;
    if (x.tiles > 0) {
      join_stats(p, x, stats, R, L);
    } else {
      if (threadIdx.x < kRows) {
        R[threadIdx.x] = -INFINITY;
        L[threadIdx.x] = 0.f;
      }
      __syncthreads();
    }
    const float m = R[row];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (x.tiles > 0 && r < p.R) {
#pragma unroll 4
      for (int32_t c = x.c0 + sub % split; c <= x.c1; c += split) {
        const int32_t rec = x.of(c);
        const float* st = p.rec_stat + rec * 2 * kRows + row;
        const float w = st[kRows] == 0.f ? 0.f : (m == -INFINITY ? 1.f : ex2_approx(st[0] - m));
        const float4 y = *reinterpret_cast<const float4*>(p.rec_o + (static_cast<int64_t>(rec) * kRows + row) * D + 4 * lane);
        o.x = fmaf(y.x, w, o.x);
        o.y = fmaf(y.y, w, o.y);
        o.z = fmaf(y.z, w, o.z);
        o.w = fmaf(y.w, w, o.w);
      }
    }
    part[sub][lane] = o;
    __syncthreads();
    if (sub % split == 0 && r < p.R) {
      for (int i = 1; i < split; ++i) {
        const float4 y = part[sub + i][lane];
        o.x += y.x;
        o.y += y.y;
        o.z += y.z;
        o.w += y.w;
      }
      float f;
      const float all = finish_row(p, bh % p.c.Hkv, m, L[row], f);
      store_o4(o_row(p, bh, r) + 4 * lane, o, f);
      if (lane == 0) p.lse[lse_index(p, bh, r)] = all * kLn2;
    }
    return;
  }
  // ---- scores into probabilities, added to the keys' weights: kWeightKeys slots of one head
  const int64_t blk = static_cast<int64_t>(blockIdx.x) - p.join_rows;
  const int32_t chunks = static_cast<int32_t>((p.c.capacity + kWeightKeys - 1) / kWeightKeys);
  const int32_t bh = static_cast<int32_t>(blk / chunks);
  const int32_t j0 = static_cast<int32_t>(blk % chunks) * kWeightKeys;
  const Pair pair = load_pair(p, bh / p.c.Hkv, nullptr);
  if (j0 >= pair.len || pair.nq == 0) return;
  __shared__ int32_t lim[kRows];
  float w[kWeightKeys / kJoinThreads] = {};
  for (int32_t rt = 0; rt < p.row_tiles; ++rt) {
    const Records x = pair_records(p, bh, rt, pair);
    if (x.c0 != x.c1) join_stats(p, x, stats, R, L);
    else __syncthreads();
    if (threadIdx.x < kRows) {
      const int32_t r = rt * kRows + static_cast<int32_t>(threadIdx.x);
      float f, v = INFINITY;
      if (r < p.R) v = x.c0 != x.c1 ? finish_row(p, bh % p.c.Hkv, R[threadIdx.x], L[threadIdx.x], f)
                                    : p.lse[lse_index(p, bh, r)] * kLog2e;
      R[threadIdx.x] = v;
      lim[threadIdx.x] = row_limit(p, pair, r);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWeightKeys / kJoinThreads; i += 2) {  // two at a time: registers, and with them blocks an SM
      const int32_t j = j0 + i * kJoinThreads + static_cast<int32_t>(threadIdx.x);
      KeyScores<2> y;
      y.load(p, static_cast<int64_t>(bh) * p.row_tiles + rt, j, kJoinThreads, pair.len);
      y.add(j, kJoinThreads, R, lim, w + i);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kWeightKeys / kJoinThreads; ++i) {
    const int32_t j = j0 + i * kJoinThreads + static_cast<int32_t>(threadIdx.x);
    if (j < pair.len) p.c.weights[static_cast<int64_t>(bh) * p.c.capacity + j] += w[i];
  }
}

// Sizes of a call that both the workspace query and the launch use.
struct Plan {
  int row_tiles, n_cta, stride;
  bool whole;
  size_t stat_bytes, o_bytes, score_bytes;
};

Plan make_plan(const bsa_kv4_fwd_args* a) {
  Plan x;
  const int64_t R = static_cast<int64_t>(a->Hq / a->cache.Hkv) * a->T;
  x.row_tiles = static_cast<int>((R + kRows - 1) / kRows);
  const int64_t tiles = (a->cache.capacity + kTileKeys - 1) / kTileKeys;
  const int64_t pairs = static_cast<int64_t>(a->cache.B) * a->cache.Hkv * x.row_tiles;
  // (a key's weight has one writer: rows in several tiles are added up by the join)
  x.whole = tiles <= kWholeTiles && !(a->accumulate && x.row_tiles > 1) && pairs <= INT32_MAX;
  x.n_cta = static_cast<int>(x.whole ? pairs : std::min<int64_t>(pairs * tiles, static_cast<int64_t>(num_sms()) * ctas_per_sm(a->cache.D)));
  x.stride = static_cast<int>((std::min<int64_t>(R, kRows) + 1) & ~int64_t(1));
  x.stat_bytes = x.whole ? 0 : static_cast<size_t>(2 * x.n_cta) * 2 * kRows * sizeof(float);
  x.o_bytes = x.whole ? 0 : static_cast<size_t>(2 * x.n_cta) * kRows * a->cache.D * sizeof(float);
  x.score_bytes = a->accumulate ? static_cast<size_t>(pairs) * a->cache.capacity * x.stride * sizeof(float) : 0;
  return x;
}

template <int D>
bsa_status launch(const Kv4FwdParams& p, int accumulate, cudaStream_t stream) {
  auto kern = p.cap_log2 > 0.f ? kv4_fwd_kernel<D, true> : kv4_fwd_kernel<D, false>;
  const size_t smem = sizeof(FwdShared<D>);
  const bsa_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem, "set kv4 forward smem size");
  if (st != BSA_OK) return st;
  cudaError_t e = launch_kernel(kern, dim3(p.n_cta), dim3(kThreads), smem, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 forward launch");
  if (p.whole) return BSA_OK;
  const int64_t chunks = accumulate ? (p.c.capacity + kWeightKeys - 1) / kWeightKeys * p.c.B * p.c.Hkv : 0;
  e = launch_kernel(kv4_join_kernel<D>, dim3(static_cast<unsigned>(p.join_rows + chunks)), dim3(kJoinThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 join launch");
  return BSA_OK;
}

}  // namespace

bool kv4_fwd_fits(const bsa_kv4_fwd_args* a) {
  const Plan x = make_plan(a);
  const int64_t heads = static_cast<int64_t>(a->cache.B) * a->cache.Hkv;
  return heads * x.row_tiles * kRows + heads * (a->cache.capacity / kWeightKeys + 1) <= INT32_MAX;
}

size_t kv4_fwd_workspace_bytes(const bsa_kv4_fwd_args* a) {
  const Plan x = make_plan(a);
  return x.stat_bytes + x.o_bytes + x.score_bytes;
}

bsa_status kv4_fwd_launch(const bsa_kv4_fwd_args* a, float scale, cudaStream_t stream) {
  const Plan x = make_plan(a);
  Kv4FwdParams p{};
  p.c = a->cache;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.o = static_cast<__nv_bfloat16*>(a->o);
  p.lse = a->lse;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.os[i] = a->o_stride[i];
  }
  p.Hq = a->Hq;
  p.T = static_cast<int32_t>(a->T);
  p.G = a->Hq / a->cache.Hkv;
  p.R = p.G * p.T;
  p.row_tiles = x.row_tiles;
  p.lens = a->lens;
  p.q_lens = a->q_lens;
  p.scale_log2 = a->logits_soft_cap > 0.f ? scale / a->logits_soft_cap : scale * kLog2e;
  p.cap_log2 = a->logits_soft_cap > 0.f ? a->logits_soft_cap * kLog2e : 0.f;
  p.sinks = a->sinks;
  p.n_sinks = a->num_sinks;
  p.sinks_kv = a->sinks_per_kv_head ? 1 : 0;
  p.n_cta = x.n_cta;
  p.whole = x.whole ? 1 : 0;
  p.rec_stat = static_cast<float*>(a->workspace);
  p.rec_o = p.rec_stat + x.stat_bytes / sizeof(float);
  p.scores = a->accumulate ? p.rec_o + x.o_bytes / sizeof(float) : nullptr;
  p.score_stride = x.stride;
  // a block a row where a pair has many records (they are then read by all of a block), else one a pair: 4096 rows
  // of 1-2 records take 16 us by the row and 8 by the pair, 512 rows of 7 records 8 and 12
  const int64_t pairs = static_cast<int64_t>(a->cache.B) * a->cache.Hkv * x.row_tiles;
  const int64_t row_blocks = pairs * std::min<int64_t>(p.R, kRows);
  p.rows_per_block = p.n_cta >= 4 * pairs ? 1 : kRows;
  p.join_rows = static_cast<int32_t>(p.rows_per_block == 1 ? row_blocks : pairs);
  p.err = device_error_word();
  p.wait_ns = wait_limit_ns();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  return a->cache.D == 128 ? launch<128>(p, a->accumulate, stream) : launch<64>(p, a->accumulate, stream);
}

}  // namespace bsa
