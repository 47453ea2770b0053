// Attention of new tokens over a cache in pages: o = sum_j p_j v_j, p_j = exp(s_j - lse), s_j = scale q.k_j
// (capped), over the keys a token sees, or over those of them in the pages of its list.
//
// The rows that read one key head (its group's q heads times the new tokens; with lists, the group's q heads of
// one token) are the 16-row side of m16n8k16 products, keys and channels the narrow one:
//     S [16 rows, 8 keys] = Q K^T,     O [16 rows, 8 channels] += P V
// The accumulators of S are the operand P of the second product, as a sum of two bf16 numbers and so in two products: both
// operands have one type, V comes as bf16, and 8 bits of a probability alone would cost O as much as its own rounding does (error
// against 64 bits 2.0e-3 of the norm, with two terms 1.7e-3, which is the output's rounding).  One term and two: 64 x 8191
// keys 309.5 and 309.7 us, 16 ragged sequences 54.3 and 55.2, 64 of 128 to 1024 31.3 and 33.1, 64 rows of 16,384 keys 23.9 and 25.9, 128
// rows 52.2 and 58.9.
// The memory bounds it by far (G rows a head: 4 G operations for 4 bytes of a key's channel); at 4 rows a head the
// products, 8 cycles each of a sub-partition, take a quarter of the time that the keys take to come.  Many rows a head (a prompt's
// tokens behind a cached prefix) read the keys again for every 64 rows and are bound by the products and the softmax between them:
// 512 tokens of 32 q heads behind 8192 keys on 8 heads 378 us, 188 TFLOP/s.
//
// A unit of loading is 16 keys (K and V), which lie in one page.  They go by 16-byte asynchronous copies, which
// take any stride between tokens, heads and pages and can bring zeros for keys that no row sees, into a ring of stages that
// belongs to the RT warps that share these keys: RT row tiles of 16, a warp each (RT = 1: a warp has its keys for itself, and
// no barrier).  A CTA's groups of RT warps take 16 keys in turn.  A group's page numbers come 32 units at a
// time, one a lane, a batch ahead.
//
// Work: all pairs (sequence, head, row tiles; with lists also token) and their tiles of 64 keys, and kPartUnits more units for
// each pair, form one sequence, cut into equal runs, one per CTA; lengths are read on the device.  A run's parts
// of pairs that other CTAs share go to the workspace as (m, l, O) records, which a second kernel joins in a fixed order.
// Where there are pairs enough, a pair goes whole to a CTA instead, and nothing is joined.
//
// 64 sequences of 8191 keys on 8 heads, 32 q heads: 309 us, 2.1 GB at 6.9 TB/s, what a copy reaches.  One sequence of 65,536 keys:
// 47 us (5.7 TB/s); 5 of them until the first keys are there (lengths, table, keys: a chain of loads), 5 the join.
#include <cmath>

#include "internal.h"
#include "paged.cuh"

namespace bsa {
namespace {

constexpr int kUnit = 16;       // keys of one load
constexpr int kTileKeys = 64;
constexpr int kRowTile = 16;
// Cost of a part beside its tiles', in tiles: lookups, the first keys' way in, the sums' way out.  3, 11 and 15 of them: 16 ragged
// sequences of up to 8192 keys on 8 heads 56.2, 54.8 and 56.5 us, 20 of them 67.6, 66.8 and 67.3, 4 of 8192 28.1, 27.1 and 27.0;
// 8 of 16,384 with 128 rows a head 57.9, 58.9 and 59.4.
constexpr int kPartUnits = 11;
// Pairs that one CTA takes alone (no records, no join), by the longest that one can be, in tiles: up to 8; up to 32 where
// there are pairs enough (tiles x SMs up to 96 x pairs; with several row tiles pairs for three quarters of the SMs); and
// lists and windows, whose lengths differ less, of up to 64 where there are pairs for half of the SMs.
// Sequences of keys on 8 heads, whole and cut (us): 16 of 2048 24.5 and 28.7, 64 of 128 to 1024 33.2 and 38.4, 6 of 1024 12.7 and
// 14.1, 6 of 2048 19.9 and 17.3, 1 of 1024 11.8 and 8.9; on one head of 64 rows 128 of 2048 57.9 and 70.3, 64 of 1024
// 33.7 and 30.1.  (One sequence of 4096 among 15 short ones would take 34 whole and takes 17.)
// Lists of 64 pages of 64, with their selection, for 64, 80, 96 and 128 pairs: 44.1 and 39.3, 47.1 and 46.9, 47.5 and 51.3, 56.5 and
// 60.6; of 40 pages, 80 and 128 pairs, 36.2 and 37.8, 42.3 and 46.6.  Windows of 2500 keys, 64, 80 and 128 pairs: 23.7 and 21.9, 23.8 and
// 24.8, 28.7 and 32.9; of 4000 34.0 and 28.4, 34.1 and 33.0, 42.4 and 46.6.
// What a pair can be is known from the table's width, not from the lengths: in a table of 8192 tokens the 16 of 2048 keys take 28.7 us
// and the 64 short ones 39.9 instead of 35.2, in one of their own width.
constexpr int kWholeTiles = 8, kManyTiles = 32, kEvenTiles = 64;
constexpr int kSmWarps = 8;      // warps an SM: a CTA of all of them, or two of four where pairs are whole to a CTA and more than SMs
constexpr int kWarpRing = 24 * 1024;
constexpr int smem_bytes(int warps) { return warps * kWarpRing + 256; }
constexpr int32_t kNoKeys = -4096;  // place of a unit without keys: before every key a row sees
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994530942f;

struct FwdParams {
  bsa_paged_cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int64_t qs[3], os[3];
  uint32_t k8[3], v8[3];  // the cache's strides, in 16 bytes
  const int32_t *table, *lens, *q_lens, *select;
  int32_t B, Hq, Hkv, T, G, shift, pages;
  int64_t M;
  int32_t keep;
  int32_t queries;    // query sets of a sequence that have keys of their own: T with lists, else 1
  int32_t R;          // rows of a pair: G * T, with lists G
  int32_t row_tiles;  // pairs of a query set and head
  Divisor by_t;       // of T
  int32_t kind;
  int64_t left, chunk;
  float scale_log2;   // scale * log2 e
  float by_cap;       // scale / cap, or 0
  float cap_log2;     // cap * log2 e, or 0
  const float* sinks;
  int32_t n_sinks, sinks_kv;
  int32_t n_cta;
  int32_t whole;      // CTA c takes pair c, all of it
  int32_t join_warps; // that join a row: 1 or all of a CTA
  float* rec_stat;    // [2 * n_cta][2][16 RT]: m and l of a CTA's first and last part
  float* rec_o;       // [2 * n_cta][16 RT][D]
  uint32_t* err;
};

// ------------------------------------------------------------------ walk

// A query set: what its pairs (one per head and row tile) have in common.
struct Pair {
  int32_t s;           // query set: sequence s / queries, its token s % queries (with lists)
  int32_t len, nq;     // keys held; new tokens
  int32_t lo, hi;      // keys lo .. hi - 1 are seen by some row (with lists: places in the list's pages)
  int32_t first_tile;
  int32_t tiles, units;
};

__device__ __forceinline__ int32_t first_key(const FwdParams& p, int32_t pos) {
  if (p.kind == BSA_MASK_LOCAL) return p.left < 0 || p.left >= pos ? 0 : pos - static_cast<int32_t>(p.left);
  if (p.kind == BSA_MASK_CHUNKED_CAUSAL) return p.chunk > pos ? 0 : pos - pos % static_cast<int32_t>(p.chunk);
  return 0;
}

__device__ __forceinline__ Pair load_pair(const FwdParams& p, int32_t s, uint32_t* err) {
  Pair x;
  x.s = s;
  const int32_t b = s / p.queries;
  x.len = paged_len(__ldcg(p.lens + b), p.M << p.shift, err);
  x.nq = p.q_lens ? paged_len(__ldcg(p.q_lens + b), p.T, err) : p.T;
  x.lo = 0;
  x.hi = 0;
  if (p.select) {
    const int32_t t = s % p.queries;
    const int32_t seen = t < x.nq ? max(x.len - x.nq + t + 1, 0) : 0;
    x.hi = min(p.keep, static_cast<int32_t>((static_cast<int64_t>(seen) + (1 << p.shift) - 1) >> p.shift)) << p.shift;
  } else if (x.nq > 0 && x.len > 0) {
    x.lo = first_key(p, max(x.len - x.nq, 0));
    x.hi = x.len;
  }
  x.first_tile = x.lo / kTileKeys;
  x.tiles = (x.hi + kTileKeys - 1) / kTileKeys - x.first_tile;
  if (x.hi == 0) x.tiles = 0;
  x.units = x.tiles > 0 ? x.tiles + kPartUnits : 0;
  return x;
}

// Units of all query sets, and of the first ones up to s; every lane of the calling warp gets both.
__device__ __forceinline__ int64_t total_units(const FwdParams& p, int32_t s, int64_t* before) {
  const int lane = threadIdx.x & 31;
  const int64_t per = static_cast<int64_t>(p.Hkv) * p.row_tiles;
  int64_t sum = 0, head = 0;
  for (int32_t i = lane; i < p.B * p.queries; i += 32) {
    const int64_t n = load_pair(p, i, nullptr).units * per;
    sum += n;
    if (i < s) head += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    head += __shfl_xor_sync(0xffffffffu, head, o);
  }
  *before = head;
  return sum;
}

// Of n runs, CTA c has units [c * total / n, (c + 1) * total / n); cta_of is the one that has unit t.
// A pair's first kPartUnits units are no tiles.
__device__ __forceinline__ int32_t runs(const FwdParams& p, int64_t total) {
  return static_cast<int32_t>(min(static_cast<int64_t>(p.n_cta), total));
}
// Of non-negative numbers, mostly small ones.  (Out of line: a kernel's first instructions come out of a cold cache.)
__device__ __noinline__ int64_t quotient64(int64_t a, int64_t b) { return a / b; }
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : quotient64(a, b);
}
__device__ __forceinline__ int64_t first_unit(int64_t c, int64_t total, int32_t n) { return quotient(c * total, n); }
__device__ __forceinline__ int32_t cta_of(int64_t t, int64_t total, int32_t n) {
  return static_cast<int32_t>(quotient((t + 1) * n - 1, total));
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int64_t scan(int64_t x) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// Cursor over a CTA's run: parts of pairs, each a range of key tiles.
struct Run {
  int64_t at, end;     // units of the run still to go
  int64_t seq0;        // first unit of query set pair.s
  Pair pair;
  int32_t h, rt;
  int32_t k0, k1;      // the part's key tiles
  bool whole;          // the part is the whole pair
  // run c of those that the query sets' units are cut into (warp-collective)
  __device__ __forceinline__ void init(const FwdParams& p, int32_t c, uint32_t* err) {
    const int lane = threadIdx.x & 31;
    const int64_t per = static_cast<int64_t>(p.Hkv) * p.row_tiles;
    const int32_t n_sets = p.B * p.queries;
    Pair x{};
    int64_t total = 0, inc = 0, own = 0;
    // up to 32 sets: a lane holds its own from here on
    for (int32_t s0 = 0; s0 < n_sets; s0 += 32) {
      x.units = 0;
      if (s0 + lane < n_sets) x = load_pair(p, s0 + lane, err);
      own = x.units * per;
      inc = scan(own);
      total += __shfl_sync(0xffffffffu, inc, 31);
    }
    const int32_t n = runs(p, total);
    at = c < n ? first_unit(c, total, n) : 0;
    end = c < n ? first_unit(c + 1, total, n) : 0;
    seq0 = 0;
    if (at >= end) return;
    for (int32_t s0 = 0;; s0 += 32) {
      if (n_sets > 32) {
        x.units = 0;
        if (s0 + lane < n_sets) x = load_pair(p, s0 + lane, nullptr);
        own = x.units * per;
        inc = scan(own);
      }
      const uint32_t past = __ballot_sync(0xffffffffu, seq0 + inc > at);
      if (past || s0 + 32 >= n_sets) {
        const int l = past ? __ffs(past) - 1 : 31;
        seq0 += __shfl_sync(0xffffffffu, inc - own, l);
        pair.s = __shfl_sync(0xffffffffu, x.s, l);
        pair.len = __shfl_sync(0xffffffffu, x.len, l);
        pair.nq = __shfl_sync(0xffffffffu, x.nq, l);
        pair.lo = __shfl_sync(0xffffffffu, x.lo, l);
        pair.hi = __shfl_sync(0xffffffffu, x.hi, l);
        pair.first_tile = __shfl_sync(0xffffffffu, x.first_tile, l);
        pair.tiles = __shfl_sync(0xffffffffu, x.tiles, l);
        pair.units = __shfl_sync(0xffffffffu, x.units, l);
        return;
      }
      seq0 += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  __device__ __forceinline__ void init_whole(const FwdParams& p, int32_t c, uint32_t* err) {
    rt = c % p.row_tiles;
    h = c / p.row_tiles % p.Hkv;
    pair = load_pair(p, c / p.row_tiles / p.Hkv, err);
    at = -1;
  }
  __device__ bool next(const FwdParams& p) {
    if (p.whole) {
      if (at == 0) return false;
      at = 0;
      k0 = pair.first_tile;
      k1 = k0 + pair.tiles;
      whole = true;
      return true;
    }
    const int64_t per = static_cast<int64_t>(p.Hkv) * p.row_tiles;
    do {
      if (at >= end) return false;
      while (at >= seq0 + pair.units * per) {
        seq0 += pair.units * per;
        pair = load_pair(p, pair.s + 1, nullptr);
      }
      const int64_t i = at - seq0;
      const int32_t hr = static_cast<int32_t>(quotient(i, pair.units));
      h = hr / p.row_tiles;
      rt = hr % p.row_tiles;
      const int32_t u0 = static_cast<int32_t>(i - static_cast<int64_t>(hr) * pair.units);
      const int32_t u1 = static_cast<int32_t>(min(static_cast<int64_t>(pair.units), u0 + (end - at)));
      at += u1 - u0;
      k0 = max(u0 - kPartUnits, 0);
      k1 = max(u1 - kPartUnits, 0);
    } while (k0 >= k1);
    whole = k0 == 0 && k1 == pair.tiles;
    k0 += pair.first_tile;
    k1 += pair.first_tile;
    return true;
  }
};

// Row r of a pair: q head and token.
__device__ __forceinline__ int32_t row_head(const FwdParams& p, int32_t h, int32_t r) { return h * p.G + (p.select ? r : p.by_t.of(r)); }
__device__ __forceinline__ int32_t row_token(const FwdParams& p, int32_t s, int32_t r) { return p.select ? s % p.queries : r - p.by_t.of(r) * p.T; }

// ------------------------------------------------------------------ loads and products

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool valid, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The RT warps that share keys.
template <int RT>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (RT == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(RT * 32) : "memory");
}

template <int D, int RT, int W>
struct FwdShared {
  static constexpr int kGroups = W / RT;
  static constexpr int kPer = RT == 1 ? 1 : 2;           // units of a step (two where the ring has room for them)
  static constexpr int kUnitBytes = kUnit * D * 2 * 2;   // K, then V
  static constexpr int kStageBytes = kPer * kUnitBytes;
  static constexpr int kStages = RT * kWarpRing / kStageBytes;
  static constexpr int kPad = D + 4;  // floats between rows of the merge buffer
  static_assert(W * kRowTile * kPad * 4 <= W * kWarpRing, "the merge buffer is the ring's memory");
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap tanh(x) of x = score / cap, in log2 units.  1 - 2 / (1 + e^2x) is off by 2^-20.8 whatever x (the exponential goes to 0 or to infinity,
// NaN stays), so it serves from 1/4 on; below, where its difference would cancel, the score times tanh(x) / x = 1 - x^2 / 3 + ..,
// the next term of which is below 2^-26.  So a cap of any size costs a score no more than its own last bits.  (64 rows of up to 16,384 keys,
// caps of 30 and 2: 25.3 and 26.9 us, the first form alone 24.9 and 25.0; with 4 rows a head within 1%.)
constexpr float kNearCap = 0.25f;
__device__ __forceinline__ float below_cap(float score_log2, float x) {
  const float y = x * x;
  const float t = fmaf(fmaf(fmaf(62.f / 2835.f, y, -17.f / 315.f), y, 2.f / 15.f), y, -1.f / 3.f);
  return fmaf(score_log2 * y, t, score_log2);
}
__device__ __forceinline__ float at_cap(float cap_log2, float x) {
  return cap_log2 * fmaf(-2.f, rcp_approx(1.f + ex2_approx(x * (2.f * kLog2e))), 1.f);
}

// Adds a row's sinks: (m, l) -> its logsumexp in log2 units and the factor of the unnormalised output.
__device__ __forceinline__ float finish_row(const FwdParams& p, int32_t h, float m, float l, float& factor) {
  float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
  factor = l == 0.f ? 0.f : 1.f / l;
  if (p.n_sinks > 0) {
    const float* z = p.sinks + (p.sinks_kv ? h * p.n_sinks : 0);
    float top = lse2;
    for (int j = 0; j < p.n_sinks; ++j) top = fmaxf(top, z[j] * kLog2e);
    float sum = lse2 == -INFINITY ? 0.f : ex2_approx(lse2 - top);
    for (int j = 0; j < p.n_sinks; ++j) sum += ex2_approx(fmaf(z[j], kLog2e, -top));
    const float all = top == -INFINITY ? -INFINITY : top + log2f(sum);
    if (l != 0.f) factor *= ex2_approx(lse2 - all);
    lse2 = all;
  }
  return lse2;
}

__device__ __forceinline__ void store_row4(const FwdParams& p, int32_t s, int32_t h, int32_t r, int d, const float4& x, float m, float l) {
  const int32_t b = s / p.queries, hq = row_head(p, h, r), t = row_token(p, s, r);
  float f;
  const float lse2 = finish_row(p, h, m, l, f);
  // (a row without keys has O = 0, whatever the keys that others see)
  const float4 y = l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
  *reinterpret_cast<uint2*>(p.o + b * p.os[0] + hq * p.os[1] + t * p.os[2] + d) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
  if (d == 0) p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.T + t] = lse2 * kLn2;
}

// Which of 16 value rows hold an infinity or a NaN, as bits.
template <int D>
__device__ __forceinline__ uint32_t odd_keys(uint32_t v, int lane) {
  bool odd = false;
  const int row = lane & 15;
#pragma unroll
  for (int x = 0; x < D / 16; ++x) {
    const int u = x + (lane >> 4) * (D / 16);
    uint32_t w[4];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(v + row * D * 2 + ((u ^ (row & 7)) << 4))
                 : "memory");
#pragma unroll
    for (int y = 0; y < 4; ++y) odd |= (w[y] & 0x7F80u) == 0x7F80u || (w[y] & 0x7F800000u) == 0x7F800000u;
  }
  const uint32_t keys = __ballot_sync(0xffffffffu, odd);
  return (keys | keys >> 16) & 0xFFFFu;
}

// Probabilities a and b as sums of two bf16 numbers, the operands of two products: the first is a (1 - 2^-8) cut to 8 bits, the second the
// rest, rounded, so 2^-14 of a are lost.  Neither is 0 where a is above 2^-125 (an infinite value stays one).
__device__ __forceinline__ void two_terms(float a, float b, uint32_t& first, uint32_t& rest) {
  const uint32_t x = __float_as_uint(a * (1.f - 0x1p-8f)), y = __float_as_uint(b * (1.f - 0x1p-8f));
  first = __byte_perm(x, y, 0x7632);
  rest = pack_bf16x2(a - __uint_as_float(x & 0xFFFF0000u), b - __uint_as_float(y & 0xFFFF0000u));
}

// O += p v of the marked keys, for the rows that see them (probabilities as the products' operands).
template <int D>
__device__ __forceinline__ void add_odd_keys(float (&acc)[D / 8][4], const uint32_t (&pa)[4], const uint32_t (&pb)[4], uint32_t keys, uint32_t v, int lane, int32_t pos,
                                          const int32_t (&lo)[2], const int32_t (&hi)[2]) {
  const int t4 = lane & 3;
  for (; keys; keys &= keys - 1) {
    const int j = __ffs(keys) - 1, from = (lane & 28) | ((j & 7) >> 1);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t w0 = __shfl_sync(0xffffffffu, i ? pb[r] : pa[r], from), w1 = __shfl_sync(0xffffffffu, i ? pb[2 + r] : pa[2 + r], from);
        const uint32_t w = j < 8 ? w0 : w1;
        x += __uint_as_float(j & 1 ? w & 0xFFFF0000u : w << 16);
      }
      if (pos + j < lo[r] || pos + j > hi[r]) continue;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint32_t y;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(y) : "r"(v + j * D * 2 + ((c ^ (j & 7)) << 4) + t4 * 4) : "memory");
        acc[c][2 * r] = fmaf(x, __uint_as_float(y << 16), acc[c][2 * r]);
        acc[c][2 * r + 1] = fmaf(x, __uint_as_float(y & 0xFFFF0000u), acc[c][2 * r + 1]);
      }
    }
  }
}

template <int D, int RT, int W, bool kCap>
__global__ void __launch_bounds__(32 * W, kSmWarps / W) paged_fwd_kernel(const __grid_constant__ FwdParams p) {
  using Sh = FwdShared<D, RT, W>;
  constexpr int kStages = Sh::kStages, kGroups = Sh::kGroups, kPer = Sh::kPer, kK = D / 16, kRows = kRowTile * RT;
  extern __shared__ uint8_t raw[];
  uint8_t* const ring = raw + (-smem_u32(raw) & 255u);  // (addresses in it are XORed below bit 8)
  __shared__ float stat_m[kGroups][kRows], stat_l[kGroups][kRows];
  __shared__ int32_t place[kGroups][kStages][kPer];  // position of a unit's first key, or kNoKeys
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile = warp % RT, group = warp / RT;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t ring0 = smem_u32(ring) + group * kStages * Sh::kStageBytes;
  griddep_wait();
  griddep_launch_dependents();  // (after the wait: the join's CTAs read the lengths at once)
  // keys and values are read once and leave the second-level cache first: tables, records and the next kernels' code stay
  // (16 ragged sequences 58 -> 56 us, an eighth of 16 x 32,768 keys 63.5 -> 60.3 us, with the selection before it)
  const uint64_t once = policy_evict_first();
  Run run;
  if (p.whole) {
    run.init_whole(p, static_cast<int32_t>(blockIdx.x), threadIdx.x == 0 ? p.err : nullptr);
  } else {
    run.init(p, static_cast<int32_t>(blockIdx.x), blockIdx.x == 0 && warp == 0 ? p.err : nullptr);
  }
  const int page_units = p.shift - 4;  // log2 of the units in a page
  int part = 0;
  for (; run.next(p); ++part) {
    const Pair& pair = run.pair;
    const int32_t b = pair.s / p.queries, h = run.h;
    const int32_t* table = p.table + b * p.M;
    const int32_t* list = p.select ? p.select + ((static_cast<int64_t>(b) * p.Hkv + h) * p.T + pair.s % p.queries) * p.keep : nullptr;
    // ---- units of this group: numbers u0 + i * kGroups, none of them before the first key that is seen or past the last
    // (the table's entries there need not be pages)
    const int32_t u0 = max(run.k0 * (kTileKeys / kUnit), pair.lo / kUnit) + group;
    const int32_t u1 = min(run.k1 * (kTileKeys / kUnit), (pair.hi + kUnit - 1) / kUnit);
    const int32_t n = u1 > u0 ? (u1 - u0 + kGroups - 1) / kGroups : 0;
    // pages of units i0 .. i0 + 31, one a lane: its number in the cache (-1: none), and in the sequence
    auto look_up = [&](int32_t i0, int32_t& page, int32_t& own) {
      page = -1;
      own = 0;
      const int32_t i = i0 + lane;
      if (i >= n) return;
      own = (u0 + i * kGroups) >> page_units;
      if (list) {
        own = list[own];
        const int32_t last = pair.len - pair.nq + pair.s % p.queries;  // (the query's position)
        if (own < 0 || own > last >> p.shift) {
          if (p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
          own = 0;
          return;
        }
      }
      page = table[own];
      if (page < 0 || page >= p.pages) {
        if (p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
        page = -1;
      }
    };
    int32_t page_now, own_now, page_next, own_next;
    look_up(0, page_now, own_now);
    look_up(32, page_next, own_next);
    // keys of a sequence that some row sees; with lists those up to the query
    const int32_t load_lo = p.select ? 0 : pair.lo, load_hi = p.select ? pair.len - pair.nq + pair.s % p.queries + 1 : pair.hi;
    // ---- copies: a lane has 16 bytes of every kStep-th row, from row0 on; the chunks of a row are XORed with its number
    constexpr int kLanes = D / 8, kStep = 32 / kLanes * RT;
    const int row0 = tile * (32 / kLanes) + lane / kLanes;
    const uint4* lane_k = static_cast<const uint4*>(p.c.k) + h * static_cast<int64_t>(p.k8[1]) + row0 * static_cast<int64_t>(p.k8[2]) + lane % kLanes;
    const uint4* lane_v = static_cast<const uint4*>(p.c.v) + h * static_cast<int64_t>(p.v8[1]) + row0 * static_cast<int64_t>(p.v8[2]) + lane % kLanes;
    const uint32_t lane_dst = ring0 + row0 * D * 2 + ((lane % kLanes ^ (row0 & 7)) << 4);
    const int32_t steps = (n + kPer - 1) / kPer;
    auto issue = [&](int32_t step, int stage) {
      if (step < steps) {
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
          const int32_t i = step * kPer + y;  // (one past the last: no page)
          const int32_t page = __shfl_sync(0xffffffffu, page_now, i & 31), own = __shfl_sync(0xffffffffu, own_now, i & 31);
          const int32_t in_page = ((u0 + i * kGroups) << 4) & ((1 << p.shift) - 1);
          const int32_t pos = (own << p.shift) + in_page;
          if (lane == 0 && tile == 0) place[group][stage][y] = page < 0 ? kNoKeys : pos;
          const uint32_t dst = lane_dst + stage * Sh::kStageBytes + y * Sh::kUnitBytes;
          const uint32_t some = BSA_RANGE(page < 0 ? 0 : page, 0, p.pages, p.err);
          const uint4* k = lane_k + (static_cast<uint64_t>(some) * p.k8[0] + static_cast<uint64_t>(in_page) * p.k8[2]);
          const uint4* v = lane_v + (static_cast<uint64_t>(some) * p.v8[0] + static_cast<uint64_t>(in_page) * p.v8[2]);
          if (page >= 0 && pos >= load_lo && pos + kUnit <= load_hi) {
#pragma unroll
            for (int x = 0; x < kUnit / kStep; ++x) {
              const uint32_t at = (dst ^ ((x * kStep & 7) << 4)) + x * kStep * D * 2;
              copy16(at, k, true, once);
              copy16(at + kUnit * D * 2, v, true, once);
              k += static_cast<uint64_t>(p.k8[2]) * kStep;
              v += static_cast<uint64_t>(p.v8[2]) * kStep;
            }
          } else {
#pragma unroll
            for (int x = 0; x < kUnit / kStep; ++x) {
              const uint32_t at = (dst ^ ((x * kStep & 7) << 4)) + x * kStep * D * 2;
              const int32_t j = pos + x * kStep + row0;
              const bool valid = page >= 0 && j >= load_lo && j < load_hi;
              copy16(at, k, valid, once);
              copy16(at + kUnit * D * 2, v, valid, once);
              k += static_cast<uint64_t>(p.k8[2]) * kStep;
              v += static_cast<uint64_t>(p.v8[2]) * kStep;
            }
          }
          if ((i & 31) == 31) {
            page_now = page_next;
            own_now = own_next;
            look_up(i + 33, page_next, own_next);
          }
        }
      }
      copy_commit();
    };
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    // ---- q by way of the ring's last stage (free until the first step), then the first stages
    const uint32_t q_at = ring0 + (kStages - 1) * Sh::kStageBytes + tile * kRowTile * D * 2;
#pragma unroll 1
    for (int x = 0; x < kRowTile * kLanes / 32; ++x) {
      const int row = x * (32 / kLanes) + lane / kLanes;
      const int32_t r = run.rt * kRows + tile * kRowTile + row, rr = min(r, p.R - 1);
      const __nv_bfloat16* src = p.q + b * p.qs[0] + row_head(p, h, rr) * p.qs[1] + row_token(p, pair.s, rr) * p.qs[2] + lane % kLanes * 8;
      copy16(q_at + row * D * 2 + ((lane % kLanes ^ (row & 7)) << 4), src, r < p.R);
    }
    copy_commit();
    // this thread's two rows: the keys they see
    int32_t lo[2], hi[2];
    bool real[2] = {false, false};  // (others' sums are not used)
    int32_t all_lo = 0, all_hi = INT32_MAX;  // keys that every row of the tile sees
    uint32_t qa[kK][4];
    // fragments: row lane & 7 (+ 8) of a matrix, its 16-byte chunks 2 k (+ 1), as XOR of the lane's first address
    const uint32_t lane_kf = ring0 + ((lane & 7) + (lane >> 4) * 8) * D * 2 + (((lane >> 3 & 1) ^ (lane & 7)) << 4);
    const uint32_t lane_vf = ring0 + kUnit * D * 2 + (lane & 15) * D * 2 + (((lane >> 4) ^ (lane & 7)) << 4);
    int stage = 0, stage_in = 0;
    // (the first kStages - 1 turns only load: one copy of the loading code, out of a cold instruction cache)
#pragma unroll 1
    for (int32_t i = 1 - kStages; i < steps; ++i) {
      if (i >= 0) {
        copy_wait<kStages - 2>();
        if (i == 0) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < kK; ++k) ldsm4(qa[k], q_at + (lane & 15) * D * 2 + ((2 * k + (lane >> 4) ^ (lane & 7)) << 4));
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int32_t rr = run.rt * kRows + tile * kRowTile + g + 8 * r, t = row_token(p, pair.s, rr);
            const int32_t at = pair.len - pair.nq + t;
            real[r] = rr < p.R && t < pair.nq && at >= 0;
            hi[r] = real[r] ? at : -1;
            lo[r] = real[r] ? first_key(p, at) : 0;
            if (real[r]) {
              all_lo = max(all_lo, lo[r]);
              all_hi = min(all_hi, hi[r]);
            }
          }
          all_lo = __reduce_max_sync(0xffffffffu, all_lo);
          all_hi = __reduce_min_sync(0xffffffffu, all_hi);
        }
        group_sync<RT>(group);
      }
      issue(i + kStages - 1, stage_in);
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
      if (i < 0) continue;
      const uint32_t at = stage * Sh::kStageBytes;
      int32_t pos[kPer];
      bool any = false, masked = false;
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        pos[y] = place[group][stage][y];
        any |= pos[y] != kNoKeys;
        masked |= pos[y] < all_lo || pos[y] + kUnit - 1 > all_hi;
      }
      stage = stage + 1 == kStages ? 0 : stage + 1;
      if (!any) continue;  // (uniform over the group)
      // ---- scores of 16 keys: element (row g + 8 (e / 2), key 8 c + 2 t4 + e % 2) is s[.][c][e]
      float s[kPer][2][4] = {};
#pragma unroll
      for (int k = 0; k < kK; ++k)
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
          uint32_t kb[4];
          ldsm4(kb, (lane_kf + at + y * Sh::kUnitBytes) ^ (k << 5));
          mma_bf16(s[y][0], qa[k], kb[0], kb[1]);
          mma_bf16(s[y][1], qa[k], kb[2], kb[3]);
        }
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        float x[2][4];
        bool far = false;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[c][e] = s[y][c][e] * p.by_cap;
            s[y][c][e] *= p.scale_log2;
            if constexpr (kCap) {
              s[y][c][e] = below_cap(s[y][c][e], x[c][e]);
              far |= !(fabsf(x[c][e]) < kNearCap);
            }
          }
        if (kCap && __any_sync(0xffffffffu, far)) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(fabsf(x[c][e]) < kNearCap)) s[y][c][e] = at_cap(p.cap_log2, x[c][e]);
        }
      }
      if (masked) {
#pragma unroll
        for (int y = 0; y < kPer; ++y)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int32_t j = pos[y] + 8 * c + 2 * t4 + (e & 1);
              if (j < lo[e >> 1] || j > hi[e >> 1]) s[y][c][e] = -INFINITY;
            }
      }
      // ---- running maximum and sum.  (A reference that lags by up to 2^8 saved the scaling of O, 1% of the time, while a
      // probability was one bf16 term, whose error it raised from 2.0e-3 to 2.4e-3 of the norm of O; with two it was not measured.)
      float top[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float x = fmaxf(fmaxf(s[0][0][2 * r], s[0][0][2 * r + 1]), fmaxf(s[0][1][2 * r], s[0][1][2 * r + 1]));
        if constexpr (kPer == 2) x = fmaxf(x, fmaxf(fmaxf(s[1][0][2 * r], s[1][0][2 * r + 1]), fmaxf(s[1][1][2 * r], s[1][1][2 * r + 1])));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        top[r] = fmaxf(m[r], fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)));
        moved |= top[r] > m[r];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          // (0 of a row's first keys; 1 for a row that has not moved: no row's bits depend on what others see)
          const float f = ex2_approx(m[r] - (top[r] == -INFINITY ? 0.f : top[r]));
          l[r] *= f;
          m[r] = top[r];
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            acc[c][2 * r] *= f;
            acc[c][2 * r + 1] *= f;
          }
        }
      }
      const float from[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float a = ex2_approx(s[y][c][2 * r] - from[r]), b = ex2_approx(s[y][c][2 * r + 1] - from[r]);
            l[r] += a + b;
            two_terms(a, b, pa[2 * c + r], pb[2 * c + r]);
          }
        const uint32_t vs = lane_vf + at + y * Sh::kUnitBytes;
        if (masked && p.T > 1 && !p.select) {
          // a key that only some rows see must not reach the others, even with values that are not numbers (0 times
          // them is not 0): such keys leave the product and are added row by row
          const uint32_t keys = odd_keys<D>(ring0 + at + y * Sh::kUnitBytes + kUnit * D * 2, lane);
          if (keys) {
            add_odd_keys<D>(acc, pa, pb, keys, ring0 + at + y * Sh::kUnitBytes + kUnit * D * 2, lane, pos[y], lo, hi);
            const uint32_t keep[2] = {(keys >> (2 * t4) & 1u ? 0u : 0xFFFFu) | (keys >> (2 * t4 + 1) & 1u ? 0u : 0xFFFF0000u),
                                      (keys >> (8 + 2 * t4) & 1u ? 0u : 0xFFFFu) | (keys >> (9 + 2 * t4) & 1u ? 0u : 0xFFFF0000u)};
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              uint32_t vb[4];
              ldsm4t(vb, vs ^ (c << 5));
#pragma unroll
              for (int x = 0; x < 4; ++x) vb[x] &= keep[x & 1];
              mma_bf16(acc[2 * c], pa, vb[0], vb[1]);
              mma_bf16(acc[2 * c + 1], pa, vb[2], vb[3]);
              mma_bf16(acc[2 * c], pb, vb[0], vb[1]);
              mma_bf16(acc[2 * c + 1], pb, vb[2], vb[3]);
            }
            continue;
          }
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t vb[4];
          ldsm4t(vb, vs ^ (c << 5));
          mma_bf16(acc[2 * c], pa, vb[0], vb[1]);
          mma_bf16(acc[2 * c + 1], pa, vb[2], vb[3]);
          mma_bf16(acc[2 * c], pb, vb[0], vb[1]);
          mma_bf16(acc[2 * c + 1], pb, vb[2], vb[3]);
        }
      }
    }
    copy_wait<0>();
    // ---- the groups' sums together
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t4 == 0) {
        stat_m[group][tile * kRowTile + g + 8 * r] = real[r] ? m[r] : -INFINITY;
        stat_l[group][tile * kRowTile + g + 8 * r] = real[r] ? l[r] : 0.f;
      }
    }
    __syncthreads();  // (and every warp is done with the ring)
    float* merge = reinterpret_cast<float*>(ring);
    const int32_t live = min(kRows, p.R - run.rt * kRows);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = tile * kRowTile + g + 8 * r;
      if (row >= live) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kGroups; ++w) top = fmaxf(top, stat_m[w][row]);
      const float f = m[r] == -INFINITY ? (l[r] == 0.f ? 0.f : 1.f) : ex2_approx(m[r] - top);
#pragma unroll
      for (int c = 0; c < D / 8; ++c)
        *reinterpret_cast<float2*>(&merge[(group * kRows + row) * Sh::kPad + 8 * c + 2 * t4]) = make_float2(acc[c][2 * r] * f, acc[c][2 * r + 1] * f);
    }
    __syncthreads();
    const int64_t rec = 2 * static_cast<int64_t>(BSA_RANGE(static_cast<int32_t>(blockIdx.x), 0, p.n_cta, p.err)) + (part > 0 ? 1 : 0);
    for (int i = threadIdx.x; i < live * (D / 4); i += 32 * W) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kGroups; ++w) top = fmaxf(top, stat_m[w][row]);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kGroups; ++w) {
        const float lw = stat_l[w][row];
        if (lw == 0.f) continue;  // (no keys)
        sum += lw * (stat_m[w][row] == -INFINITY ? 1.f : ex2_approx(stat_m[w][row] - top));
        const float4 y = *reinterpret_cast<const float4*>(&merge[(w * kRows + row) * Sh::kPad + d]);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      if (run.whole) {
        store_row4(p, pair.s, h, run.rt * kRows + row, d, x, top, sum);
      } else {
        *reinterpret_cast<float4*>(p.rec_o + (rec * kRows + row) * D + d) = x;
        if (d == 0) {
          p.rec_stat[rec * 2 * kRows + row] = top;
          p.rec_stat[rec * 2 * kRows + kRows + row] = sum;
        }
      }
    }
    __syncthreads();  // the next part writes the ring and `stat` again
  }
}

// ------------------------------------------------------------------ join

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;

// One row of a pair, by a warp or by all of a CTA: the records of CTAs c0 .. c1, a CTA's being its first part unless its
// run began in an earlier pair (which only c0's can have).  Each warp joins some with a running maximum.
template <int D, int RT>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ FwdParams p) {
  constexpr int kRows = kRowTile * RT, kVec = D / 4, kSide = 32 / kVec;  // records side by side in a warp
  __shared__ float4 part[kJoinWarps][kVec];
  __shared__ float stats[kJoinWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int32_t rows = min(p.R, kRows);  // (a last, shorter tile has rows past its end)
  const bool wide = p.join_warps > 1;
  const int64_t at = wide ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(blockIdx.x) * kJoinWarps + warp;
  const int32_t hr = static_cast<int32_t>(at / rows), row = static_cast<int32_t>(at - static_cast<int64_t>(hr) * rows);
  const int32_t rt = hr % p.row_tiles, h = hr / p.row_tiles % p.Hkv, s = hr / p.row_tiles / p.Hkv;
  const int32_t r = rt * kRows + row;
  // Where the records are: known from the lengths, before the first kernel ends (it lets this one start once its own
  // wait is over, so what wrote the lengths has ended).
  bool mine = s < p.B * p.queries && r < p.R;  // (uniform over the warp)
  int32_t c0 = 0, c1 = -1, first = 0;
  if (mine) {
    const Pair pair = load_pair(p, s, nullptr);
    if (pair.tiles > 0) {
      int64_t before;
      const int64_t total = total_units(p, s, &before);
      const int32_t n = runs(p, total);
      const int64_t begin = before + (static_cast<int64_t>(h) * p.row_tiles + rt) * pair.units;
      c0 = cta_of(begin + kPartUnits, total, n);
      c1 = cta_of(begin + pair.units - 1, total, n);
      first = 2 * c0 + (first_unit(c0, total, n) < begin ? 1 : 0);
      mine = c0 != c1;  // else one CTA had all of it
    }
  }
  griddep_launch_dependents();
  griddep_wait();
  if (!mine) return;  // (where the CTA has one row: all of it)
  const int vec = lane % kVec;
  float m = -INFINITY, l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float mc, float lc, const float4& y) {
    if (lc == 0.f) return;  // (no keys)
    const float to = fmaxf(m, mc), from = to == -INFINITY ? 0.f : to;
    const float f = l == 0.f ? 0.f : m == -INFINITY ? 1.f : ex2_approx(m - from), fc = mc == -INFINITY ? 1.f : ex2_approx(mc - from);
    l = l * f + lc * fc;
    x.x = x.x * f + y.x * fc;
    x.y = x.y * f + y.y * fc;
    x.z = x.z * f + y.z * fc;
    x.w = x.w * f + y.w * fc;
    m = to;
  };
  const int32_t step = kSide * (wide ? kJoinWarps : 1);
  for (int32_t c = c0 + (wide ? warp * kSide : 0) + lane / kVec; c <= c1; c += 4 * step) {
    float mc[4], lc[4];
    float4 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = c + i * step <= c1;
      const int64_t rec = BSA_RANGE(!in ? first : c + i * step == c0 ? first : 2 * (c + i * step), 0, 2 * p.n_cta, p.err);
      mc[i] = p.rec_stat[rec * 2 * kRows + row];
      lc[i] = in ? p.rec_stat[rec * 2 * kRows + kRows + row] : 0.f;
      y[i] = *reinterpret_cast<const float4*>(p.rec_o + (rec * kRows + row) * D + 4 * vec);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) add(mc[i], lc[i], y[i]);
  }
#pragma unroll
  for (int o = kVec; o < 32; o *= 2) {
    const float mc = __shfl_xor_sync(0xffffffffu, m, o), lc = __shfl_xor_sync(0xffffffffu, l, o);
    const float4 y = make_float4(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o),
                                 __shfl_xor_sync(0xffffffffu, x.z, o), __shfl_xor_sync(0xffffffffu, x.w, o));
    add(mc, lc, y);
  }
  if (wide) {
    if (lane < kVec) part[warp][vec] = x;
    if (lane == 0) {
      stats[warp][0] = m;
      stats[warp][1] = l;
    }
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < kJoinWarps; ++w) add(stats[w][0], stats[w][1], part[w][vec]);
  }
  if (lane < kVec) store_row4(p, s, h, r, 4 * vec, x, m, l);
}

// Sizes of a call that both the workspace query and the launch use.
struct Plan {
  int rt;         // row tiles of a CTA
  int64_t row_tiles, pairs;
  int32_t R, n_cta;
  bool whole;
  size_t stat_bytes, o_bytes;
};

Plan make_plan(const bsa_paged_fwd_args* a) {
  Plan x;
  const int64_t G = a->Hq / a->cache.Hkv;
  x.R = static_cast<int32_t>(a->select ? G : G * a->T);
  // (8 sequences of 16,384 keys on one head, as one, two or four tiles: 16 rows 21.1, 22.9 and 31.8 us, 24 rows 27.0, 23.6 and 32.4, 32
  // rows 27.7, 24.2 and 32.7, 64 rows 40.2, 34.7 and 34.5, 128 rows 64.3, 58.8 and 58.6: tiles that share keys read them once, and
  // wait for each other)
  x.rt = x.R <= kRowTile ? 1 : x.R <= 2 * kRowTile ? 2 : 4;
  const int64_t rows = kRowTile * x.rt;
  x.row_tiles = (x.R + rows - 1) / rows;
  x.pairs = static_cast<int64_t>(a->B) * (a->select ? a->T : 1) * a->cache.Hkv * x.row_tiles;
  // the longest a pair can be: what the table, a list or a window holds
  const int64_t room = a->M * a->cache.page;
  int64_t longest = a->select ? std::min(a->keep * a->cache.page, room) : room;
  if (a->kind == BSA_MASK_LOCAL && a->local_left >= 0) longest = std::min(longest, std::min(a->local_left, room) + a->T + kTileKeys);
  if (a->kind == BSA_MASK_CHUNKED_CAUSAL) longest = std::min(longest, std::min(a->chunk, room) + a->T + kTileKeys);
  const int64_t tiles = (longest + kTileKeys - 1) / kTileKeys;
  const bool many = tiles <= kManyTiles && (x.rt == 1 ? tiles * num_sms() <= 96 * x.pairs : 4 * x.pairs >= 3 * num_sms());
  const bool even = x.rt == 1 && 2 * x.pairs >= num_sms() && tiles <= kEvenTiles && longest < room;
  x.whole = (tiles <= kWholeTiles || many || even) && x.pairs <= INT32_MAX;
  x.n_cta = static_cast<int32_t>(x.whole ? x.pairs : std::min<int64_t>(x.pairs * tiles, static_cast<int64_t>(num_sms())));
  x.stat_bytes = x.whole ? 0 : static_cast<size_t>(2 * x.n_cta) * 2 * rows * sizeof(float);
  x.o_bytes = x.whole ? 0 : static_cast<size_t>(2 * x.n_cta) * rows * a->cache.D * sizeof(float);
  return x;
}

template <int D, int RT>
bsa_status launch(const FwdParams& p, const Plan& x, cudaStream_t stream) {
  const int warps = p.whole && p.n_cta > num_sms() ? kSmWarps / 2 : kSmWarps;
  auto kern = warps < kSmWarps ? (p.cap_log2 > 0.f ? paged_fwd_kernel<D, RT, kSmWarps / 2, true> : paged_fwd_kernel<D, RT, kSmWarps / 2, false>)
                      : (p.cap_log2 > 0.f ? paged_fwd_kernel<D, RT, kSmWarps, true> : paged_fwd_kernel<D, RT, kSmWarps, false>);
  const bsa_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem_bytes(warps), "set paged forward smem size");
  if (st != BSA_OK) return st;
  cudaError_t e = launch_kernel(kern, dim3(p.n_cta), dim3(32 * warps), smem_bytes(warps), stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged forward launch");
  if (p.whole) return BSA_OK;
  const int64_t rows = x.pairs * std::min<int64_t>(p.R, kRowTile * RT), per = kJoinWarps / p.join_warps;
  e = launch_kernel(paged_join_kernel<D, RT>, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(kJoinThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged join launch");
  return BSA_OK;
}

template <int D>
bsa_status launch_rows(const FwdParams& p, const Plan& x, cudaStream_t stream) {
  return x.rt == 1 ? launch<D, 1>(p, x, stream) : x.rt == 2 ? launch<D, 2>(p, x, stream) : launch<D, 4>(p, x, stream);
}

}  // namespace

bool paged_fwd_fits(const bsa_paged_fwd_args* a) {
  const Plan x = make_plan(a);
  return x.pairs <= INT32_MAX / (kRowTile * x.rt);
}

size_t paged_fwd_workspace_bytes(const bsa_paged_fwd_args* a) {
  const Plan x = make_plan(a);
  return x.stat_bytes + x.o_bytes;
}

bsa_status paged_fwd_launch(const bsa_paged_fwd_args* a, float scale, cudaStream_t stream) {
  const Plan x = make_plan(a);
  FwdParams p{};
  p.c = a->cache;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.o = static_cast<__nv_bfloat16*>(a->o);
  p.lse = a->lse;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.os[i] = a->o_stride[i];
  }
  for (int i = 0; i < 3; ++i) {
    p.k8[i] = static_cast<uint32_t>(a->cache.k_stride[i] / 8);
    p.v8[i] = static_cast<uint32_t>(a->cache.v_stride[i] / 8);
  }
  p.table = a->table;
  p.lens = a->lens;
  p.q_lens = a->q_lens;
  p.select = a->select;
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->cache.Hkv;
  p.T = static_cast<int32_t>(a->T);
  p.G = a->Hq / a->cache.Hkv;
  p.shift = page_shift(a->cache.page);
  p.pages = static_cast<int32_t>(a->cache.pages);
  p.M = a->M;
  p.keep = a->select ? static_cast<int32_t>(a->keep) : 0;
  p.queries = a->select ? p.T : 1;
  p.R = x.R;
  p.row_tiles = static_cast<int32_t>(x.row_tiles);
  p.by_t = Divisor(static_cast<uint32_t>(p.T));
  p.kind = a->kind;
  p.left = a->local_left;
  p.chunk = a->chunk;
  p.scale_log2 = scale * kLog2e;
  p.by_cap = a->logits_soft_cap > 0.f ? scale / a->logits_soft_cap : 0.f;
  p.cap_log2 = a->logits_soft_cap > 0.f ? a->logits_soft_cap * kLog2e : 0.f;
  p.sinks = a->sinks;
  p.n_sinks = a->num_sinks;
  p.sinks_kv = a->sinks_per_kv_head ? 1 : 0;
  p.n_cta = x.n_cta;
  p.whole = x.whole ? 1 : 0;
  // (records of a pair: some n_cta / pairs.  One sequence of 65,536 keys by one warp a row 51.1 us, by eight 47.0; 64 of 4096 163 and 171)
  p.join_warps = x.n_cta >= 4 * x.pairs ? kJoinWarps : 1;
  p.rec_stat = static_cast<float*>(a->workspace);
  p.rec_o = p.rec_stat + x.stat_bytes / sizeof(float);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  return a->cache.D == 128 ? launch_rows<128>(p, x, stream) : launch_rows<64>(p, x, stream);
}

}  // namespace bsa
