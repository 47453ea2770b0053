// The attention weight every key of a prompt has received:
//   w[j] = sum over the group's q heads and the queries i that see j of exp(scale q_i.k_j - lse_i).
// The loop is the dK/dV launch's: a tile is a key block of one key head, its
// items the non-empty query blocks of each q head's row of the dkv MaskInfo.
//
// Per item one 128 x 128 x D product and 128^2 exponentials.  Keys are the
// product's M side (tensor-memory lanes), queries its columns, so a thread sums
// its key's probabilities in registers and a warpgroup can take a whole item:
// three warpgroups on three items in turn, each at another point of its item,
// keep the exponential unit busy through one another's waits.  (Queries as the
// M side leave 64 sums per thread, which forces the warpgroups onto one item
// together: they then wait, load and compute in step, 283 us on GQA 32/8 causal
// 8192, D = 128, for 194.)
//
// Shared-memory bandwidth is the other limit: both operands from shared memory
// take all of its 128 bytes a cycle while a product runs.  K therefore sits in
// tensor memory as the A operand, and a query's logsumexp enters through one
// more k-step, a tile of ones times -lse / scale in three bf16 pieces: reading
// it per column instead costs 256 cycles an item.  (With a soft cap the
// logsumexp has to be added after the tanh, and is read per column.)
//
// One persistent CTA per SM, warp-specialised:
//   warp 0      walks MaskInfo, 32 cells of a row at a time, and publishes the
//               items in a ring, several at once
//   warps 1-2   tcgen05 issuers of the even and the odd items: S^T = K Q^T into
//               one of three tensor-memory buffers (one issuer needs ~1,100
//               cycles an item, most of it barrier latency)
//   warp 3      loads Q per item and its exponent terms
//   warps 4-7   bring a tile's K from global into tensor memory (2 buffers)
//   warps 8-19  exponentials: warpgroup n % 3 takes item n
// All items of the launch form one sequence, cut into equal runs, one per CTA
// (the host computes the cuts from MaskInfo's row lengths and passes them as
// kernel parameters: no schedule to upload).  A first kernel turns the
// logsumexp into exponent terms: the producer lane, at ~1,100 cycles an item,
// set the pace while they were made beside it.  Each warpgroup leaves a row of
// sums per tile and CTA in the workspace, and a second kernel adds these up in
// order.  Neither kernel is started early (a CTA that waits for its predecessor
// holds the place of one that works: 203 us).
//
// GQA 32/8 causal 8192, D = 128: 194 us for 279 GFLOP, 1.44 PFLOP/s, in a run of tens of
// calls; 217 us at the clocks that hundreds in a row sustain.  The products
// alone would take 129 us at 512 + 64 cycles an item, the exponentials 115.  What
// is left is the barriers between the roles, ~800 cycles of issuer per two items
// and ~1,590 of warpgroup per three.  Two prompts of 4096 with a local
// window of 1024, 16 heads, D = 64: 36 us, of which 11 are the two small kernels.
// With a soft cap 1342 and 204 us: three special functions a score in place of one, the
// logsumexps read per column, and registers that spill (96 a thread).
#include <cmath>

#include "internal.h"
#include "maskinfo_dev.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace bsa {
namespace {

constexpr int kBufs = 3;        // score buffers, warpgroups of the exponentials (item n: n % 3)
constexpr int kStages = 6;      // Q and exponent terms
constexpr int kRing = 32;       // items between the walker and the producer (which reads one per lane)
constexpr int kBatch = 16;      // items published at once
constexpr int kEwWarp0 = 8;
constexpr int kEwWarps = 4 * kBufs;
constexpr int kThreads = 32 * (kEwWarp0 + kEwWarps);
constexpr int kMaxCtas = 160;
constexpr uint32_t kColK = 128 * kBufs;  // tensor memory: the score buffers, then K (2 buffers of D / 2 columns)
constexpr uint32_t kHidden = 0xFFFFDEADu;  // (a NaN no product gives) mark of an unseen score under a cap
constexpr float kLog2e = 1.4426950408889634f;

// flags of an item, beside its column (bits 0-15) and label (16-17)
constexpr uint32_t kFirst = 1u << 20;  // first item of its part of a tile
constexpr uint32_t kMask = 1u << 21;   // some pairs of the item are not visible
constexpr uint32_t kEnd = 1u << 22;    // no item: the run has ended

// A block's exponent terms: without a cap a [128 queries, 16] bf16 operand in
// 8 x 16-byte core matrices (the two k-halves of 8 rows side by side), whose
// first three columns sum to -lse / scale; with one 128 floats, -lse log2 e.
template <bool kCap>
struct Terms {
  static constexpr int kBytes = kCap ? 512 : 4096;
};

template <int D>
struct __align__(1024) KwSmem {
  static constexpr int kTileBytes = 128 * D * 2;
  uint8_t q[kStages][kTileBytes];
  uint8_t term[kStages][4096];
  uint8_t ones[4096];        // [128 keys, 16] bf16, laid out like the terms: 1 in the first three columns
  // {column | label << 16 | flags, stack slot, part of the run (tile - first tile), end of the counted queries}
  uint4 entry[kRing];
  uint2 rows[kRing];         // {Q row, K row}
  uint4 item[kStages];       // the entries, handed on
  uint32_t q_info[kStages];  // for the issuers: flags, bits 0-7 the K buffer, 8-15 the parity of its load
  uint32_t part_row[2];      // K row of the part to load, or ~0: the end
  uint64_t ring_full[kRing], ring_empty[kRing];
  // item n's stage n % kStages: q_full (Q and terms in), stage_empty (its warpgroup is done with it, Q long read)
  uint64_t q_full[kStages], stage_empty[kStages];
  uint64_t s_full[kBufs], s_empty[kBufs];
  uint64_t part_full[2], part_read[2], k_full[2];
  uint64_t drain[2];
  uint32_t tmem_base, abort_flag;
};
static_assert(sizeof(KwSmem<128>) + 1024 <= 232448, "key weights shared memory exceeds 227 KB per CTA");
static_assert(kColK + 2 * 64 <= 512, "tensor memory");

// Where a CTA's run begins: item `skip` of tile (b * Hkv + g) * rows + j.
struct Cut {
  int32_t tile, skip;
};

struct KwParams {
  int32_t B, Hq, Hkv;
  int64_t Sq, Skv;
  float scale_log2;  // without a cap scale * log2 e; with one scale / cap
  float cap_log2;
  const float* lse;
  const int32_t* q_lens;
  const __nv_bfloat16* k;
  void* terms;     // the blocks of 128 queries' exponent terms, in the order of the queries
  float term_scale, hidden;  // terms: lse * term_scale, or `hidden` for what is not counted
  float* out;
  float* sums;     // [n_tiles + 2 n_cta][kBufs][128]: a whole tile's sums of each warpgroup, then the first and last parts' of each CTA
  int32_t n_tiles;
  MaskInfoDev mi;
  int32_t compact;  // rows hold their non-empty blocks first
  int32_t n_cta;
  uint32_t* err;
  uint64_t wait_ns;
  Cut cut[kMaxCtas + 1];
};

__device__ __forceinline__ int32_t tile_items(const KwParams& p, int32_t tile) {
  const int32_t j = tile % p.mi.rows, G = p.Hq / p.Hkv;
  if (p.mi.heads == 1) return p.mi.row_len[j] * G;
  const int32_t g = tile / p.mi.rows % p.Hkv;
  int32_t n = 0;
  for (int32_t i = 0; i < G; ++i) n += p.mi.row_len[(g * G + i) * p.mi.rows + j];
  return n;
}

// Queries of sequence b that count.
__device__ __forceinline__ int32_t query_end(const KwParams& p, int32_t b) {
  return p.q_lens ? min(max(p.q_lens[b], 0), static_cast<int32_t>(p.Sq)) : static_cast<int32_t>(p.Sq);
}

// The row of sums of CTA c's part of tile t: the tile's own if c has all of it.
__device__ __forceinline__ int32_t sums_row(const KwParams& p, int32_t c, int32_t t) {
  const Cut a = p.cut[c], b = p.cut[c + 1];
  const bool whole = !(t == a.tile && a.skip > 0) && !(t == b.tile && b.skip > 0);
  return whole ? t : p.n_tiles + 2 * c + (t == a.tile ? 0 : 1);
}

// Exponent terms of all queries, one thread each.
template <bool kCap>
__global__ void __launch_bounds__(256) key_weights_terms(const __grid_constant__ KwParams p) {
  griddep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(p.B) * p.Hq * p.Sq) return;
  const float l = p.lse[i];
  const int32_t b = static_cast<int32_t>(i / (p.Hq * p.Sq)), q = static_cast<int32_t>(i % p.Sq);
  const bool gone = q >= query_end(p, b) || l == -INFINITY;
  const float t = gone ? p.hidden : l * p.term_scale;
  if constexpr (kCap) {
    static_cast<float*>(p.terms)[i] = t;
  } else {
    // three pieces of 8 bits hold all 24 of the fp32 term (hidden, or an infinity: the first alone)
    const __nv_bfloat16 hi = __float2bfloat16_rn(t);
    const float r1 = gone || isinf(__bfloat162float(hi)) ? 0.f : t - __bfloat162float(hi);
    const __nv_bfloat16 mid = __float2bfloat16_rn(r1);
    const __nv_bfloat16 lo = __float2bfloat16_rn(r1 - __bfloat162float(mid));
    uint8_t* at = static_cast<uint8_t*>(p.terms) + i / 128 * 4096 + (i % 128) / 8 * 256 + (i % 8) * 16;
    *reinterpret_cast<uint4*>(at) =
        make_uint4(static_cast<uint32_t>(__bfloat16_as_ushort(hi)) | static_cast<uint32_t>(__bfloat16_as_ushort(mid)) << 16,
                   __bfloat16_as_ushort(lo), 0u, 0u);
    *reinterpret_cast<uint4*>(at + 128) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Scores of unseen columns become what add_probs turns into an exponent of
// -infinity: an infinity of the scale's opposite sign, or (cap) a mark.
template <bool kCap>
__device__ __forceinline__ void hide(const KwParams& p, uint32_t (&v)[32], uint32_t seen) {
  const uint32_t gone = kCap ? kHidden : (p.scale_log2 > 0.f ? 0xFF800000u : 0x7F800000u);
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!(seen & (1u << i))) v[i] = gone;
}

// exp2 of one key's scores of 32 queries (less the queries' logsumexp, which
// the scores hold already, or with a cap after the terms), added to four sums.
template <bool kCap>
__device__ __forceinline__ void add_probs(const KwParams& p, const uint32_t (&v)[32], const float* term, uint64_t (&acc)[4]) {
  const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float e0, e1;
    if constexpr (kCap) {
      const float2 t = *reinterpret_cast<const float2*>(term + 2 * i);
      e0 = v[2 * i] == kHidden ? -INFINITY : fmaf(tanh_nan(__uint_as_float(v[2 * i]) * p.scale_log2), p.cap_log2, t.x);
      e1 = v[2 * i + 1] == kHidden ? -INFINITY : fmaf(tanh_nan(__uint_as_float(v[2 * i + 1]) * p.scale_log2), p.cap_log2, t.y);
    } else {
      f2_unpack(f2_mul(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2), e0, e1);
    }
    acc[i & 3] = f2_add(acc[i & 3], f2_pack(ex2_approx(e0), ex2_approx(e1)));
  }
}

// Bits of the visible queries [32 c, 32 c + 32) of the item for a key, of a masked item.
struct Visible {
  uint32_t w[4];
};
__device__ __forceinline__ Visible visible_queries(const KwParams& p, const uint4& x, int64_t key, int r) {
  Visible m{{~0u, ~0u, ~0u, ~0u}};
  const int32_t q0 = static_cast<int32_t>(x.x & 0xFFFFu) * 128;
  int64_t lo = q0, hi = static_cast<int64_t>(x.w) - 1;
  if (((x.x >> 16) & 3u) == 1u) {
    if (p.mi.kind == BSA_MASK_DENSE) {
      const uint4 bits = __ldg(reinterpret_cast<const uint4*>(p.mi.partial_bits) + static_cast<int64_t>(x.y) * 128 + r);
      m.w[0] = bits.x;
      m.w[1] = bits.y;
      m.w[2] = bits.z;
      m.w[3] = bits.w;
    } else {
      int64_t a, b;
      query_interval(p.mi.kind, p.mi.left, p.mi.right, p.mi.chunk, key, a, b);
      lo = a > lo ? a : lo;
      hi = b < hi ? b : hi;
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int64_t c0 = q0 + 32 * c;
    const int64_t a = lo > c0 ? lo - c0 : 0, b = hi < c0 + 31 ? hi - c0 : 31;
    m.w[c] &= b < a ? 0u : (0xFFFFFFFFu >> (31 - (b - a))) << a;
  }
  return m;
}

template <int D, bool kCap>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ KwParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = KwSmem<D>;
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr uint32_t kTileBytes = Smem::kTileBytes;
  const int warp = warp_id(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s.ring_full[i], 1);
      mbar_init(&s.ring_empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.stage_empty[i], 4);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.part_full[i], 1);
      mbar_init(&s.part_read[i], 4);
      mbar_init(&s.k_full[i], 4);
      mbar_init(&s.drain[i], 1);
    }
    fence_mbar_init();
  }
  if (threadIdx.x < 256) {
    const int i = threadIdx.x;  // 16 bytes of the tile of ones each
    *reinterpret_cast<uint4*>(s.ones + i * 16) = i / 8 % 2 == 0 ? make_uint4(0x3F803F80u, 0x3F80u, 0u, 0u) : make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s.tmem_base, 0);
  const WaitCtl wc{p.err, &s.abort_flag, p.wait_ns};
  griddep_wait();
  const Cut c0 = p.cut[blockIdx.x], c1 = p.cut[blockIdx.x + 1];

  if (warp == 0) {
    // ------------------------------------------------ walker (whole warp)
    uint32_t e = 0;
    bool ok = true;
    // lanes 0 .. m - 1 (in the order of `index`) publish an item each: the one
    // reader frees slots in order, so a wait for the last slot covers all
    auto room = [&](uint32_t m) -> bool {
      const uint32_t last = e + m - 1;
      return last < static_cast<uint32_t>(kRing) ||
             mbar_wait_warp(&s.ring_empty[last % kRing], (last / kRing - 1) & 1u, wc);
    };
    const int32_t G = p.Hq / p.Hkv;
    for (int32_t tile = c0.tile; ok && tile <= c1.tile; ++tile) {
      if (tile == c1.tile && c1.skip == 0) break;
      const int32_t j = tile % p.mi.rows, bg = tile / p.mi.rows, b = bg / p.Hkv, g = bg % p.Hkv;
      const int32_t all = tile_items(p, tile);
      const int32_t begin = tile == c0.tile ? c0.skip : 0;
      const int32_t stop = tile == c1.tile ? c1.skip : all;
      const int32_t q_end = query_end(p, b);
      const uint32_t krow = static_cast<uint32_t>(static_cast<int64_t>(bg) * p.Skv + static_cast<int64_t>(j) * 128);
      bool first = true;
      int32_t at = 0;  // items of the tile passed so far
      for (int32_t gh = 0; ok && gh < G && at < stop; ++gh) {
        const int32_t hq = g * G + gh, hm = p.mi.heads == 1 ? 0 : hq;
        const int32_t len = p.mi.row_len[hm * p.mi.rows + j];
        if (at + len <= begin) {
          at += len;
          continue;
        }
        const int64_t row_base = (static_cast<int64_t>(hm) * p.mi.rows + j) * p.mi.width;
        const int64_t head = (static_cast<int64_t>(b) * p.Hq + hq) * p.Sq;
        const int32_t end = min(at + len, stop);
        int32_t pos = p.compact && at < begin ? begin - at : 0;
        at += pos;
        for (; ok && at < end && pos < p.mi.width; pos += 32) {
          const RawRef raw = pos + lane < p.mi.width ? load_block(p.mi, row_base, pos + lane) : RawRef{0, 0, 0};
          const BlockRef br = check_block(p.mi, raw, p.err);
          // this lane's place among the row's items, and whether it is one to compute
          const uint32_t cells = __ballot_sync(0xffffffffu, br.label != 0);
          const int32_t mine = at + __popc(cells & ((1u << lane) - 1u));
          const bool item = br.label != 0 && mine >= begin && mine < end && br.col * 128 < q_end;  // (not padding only)
          at = min(at + __popc(cells), end);
          const uint32_t items = __ballot_sync(0xffffffffu, item);
          const uint32_t count = __popc(items), index = __popc(items & ((1u << lane) - 1u));
          for (uint32_t i0 = 0; ok && i0 < count; i0 += kBatch) {
            const uint32_t m = min(static_cast<uint32_t>(kBatch), count - i0);
            ok = room(m);
            if (!ok) break;
            if (item && index >= i0 && index < i0 + m) {
              const uint32_t slot = (e + index - i0) % kRing;
              const bool mask = br.label == 1 || br.col * 128 + 128 > q_end;
              const int64_t qrow = BSA_RANGE(head + static_cast<int64_t>(br.col) * 128, int64_t(0),
                                             static_cast<int64_t>(p.B) * p.Hq * p.Sq - 127, p.err);
              s.entry[slot] = make_uint4(static_cast<uint32_t>(br.col) | static_cast<uint32_t>(br.label) << 16 |
                                             (first && index == 0 ? kFirst : 0u) | (mask ? kMask : 0u),
                                         static_cast<uint32_t>(br.slot), static_cast<uint32_t>(tile - c0.tile),
                                         static_cast<uint32_t>(q_end));
              s.rows[slot] = make_uint2(static_cast<uint32_t>(qrow), krow);
              mbar_arrive(&s.ring_full[slot]);
            }
            __syncwarp();
            e += m;
          }
          if (count) first = false;
        }
        at = end;
      }
    }
    if (ok && room(1) && lane == 0) {
      s.entry[e % kRing] = make_uint4(kEnd, 0u, 0u, 0u);
      mbar_arrive(&s.ring_full[e % kRing]);
    }
  } else if (warp == 3) {
    // ------------------------------------------------ producer (whole warp; converged code issues copies faster than one lane's)
    if (lane == 0) tma_prefetch_desc(&tm_q);
    __syncwarp();
    const uint64_t pol = policy_evict_last();
    uint32_t n = 0, parts = 0;
    uint32_t last1 = 0, last2 = 0;  // items passed when the part before the current one, and the one before that, had ended
    bool ok = true;
    // item i's warpgroup has done with its stage (so its scores are computed); i among the last kStages items
    auto done = [&](uint32_t i) -> bool { return mbar_wait_warp(&s.stage_empty[i % kStages], (i / kStages) & 1u, wc); };
    auto stage_free = [&]() -> bool { return n < static_cast<uint32_t>(kStages) || done(n - kStages); };
    // hands the loaders a K row, or the end
    auto hand_part = [&](uint32_t row) -> bool {
      const uint32_t kb = parts & 1u;
      if (parts >= 2 && !mbar_wait_warp(&s.part_read[kb], (parts / 2 - 1) & 1u, wc)) return false;
      if (lane == 0) {
        s.part_row[kb] = row;
        mbar_arrive(&s.part_full[kb]);
      }
      __syncwarp();
      ++parts;
      return true;
    };
    // Entries are taken from the ring a batch at a time, one per lane: a wait
    // per entry, with its two reads, cost more than the copies themselves.
    uint32_t e = 0, have = 0, next = 0;  // next entry of the ring; entries at hand, and those of them passed
    uint4 mine = make_uint4(0, 0, 0, 0);
    uint2 mine_rows = make_uint2(0, 0);
    while (ok) {
      if (next == have) {
        if (!mbar_wait_warp(&s.ring_full[e % kRing], (e / kRing) & 1u, wc)) { ok = false; break; }
        const uint32_t slot = (e + lane) % kRing;
        // (kRing lanes: every slot once; a slot whose entry lies a lap ahead shows the phase before it)
        const uint32_t full = __ballot_sync(0xffffffffu, mbar_test_wait(smem_u32(&s.ring_full[slot]), ((e + lane) / kRing) & 1u));
        have = full == 0xffffffffu ? 32u : static_cast<uint32_t>(__ffs(~full) - 1);
        next = 0;
        if (static_cast<uint32_t>(lane) < have) {
          mine = s.entry[slot];
          mine_rows = s.rows[slot];
          mbar_arrive(&s.ring_empty[slot]);
        }
        __syncwarp();
        e += have;
        if (have == 0) { ok = false; break; }  // (the wait above has seen entry e)
      }
      const uint32_t st = n % kStages;
      const uint32_t flags = __shfl_sync(0xffffffffu, mine.x, next);
      if (flags & kEnd) break;
      const uint32_t qrow = __shfl_sync(0xffffffffu, mine_rows.x, next);
      const uint4 x = make_uint4(flags, __shfl_sync(0xffffffffu, mine.y, next), __shfl_sync(0xffffffffu, mine.z, next),
                                 __shfl_sync(0xffffffffu, mine.w, next));
      const uint32_t krow = __shfl_sync(0xffffffffu, mine_rows.y, next);
      ++next;
      if (!stage_free()) { ok = false; break; }
      if (flags & kFirst) {
        // the K buffer's part ended with item last2 - 1
        for (uint32_t i = n >= kStages ? n - kStages + 1 : 0; ok && parts >= 2 && i < last2; ++i) ok = done(i);
        if (!ok || !hand_part(krow)) { ok = false; break; }
        last2 = last1;
      }
      last1 = n + 1;
      const uint32_t k = parts - 1;
      if (lane == 0) {
        s.q_info[st] = (k & 1u) | ((k >> 1) & 1u) << 8;
        s.item[st] = x;
      }
      __syncwarp();
      mbar_arrive_expect_tx_elect(&s.q_full[st], kTileBytes + Terms<kCap>::kBytes);
      tma_load_3d_elect(s.q[st], &tm_q, &s.q_full[st], 0, static_cast<int32_t>(qrow), 0, pol);
      bulk_load_elect(s.term[st], static_cast<const uint8_t*>(p.terms) + static_cast<int64_t>(qrow / 128) * Terms<kCap>::kBytes,
                      Terms<kCap>::kBytes, &s.q_full[st]);
      ++n;
    }
    const uint32_t loads = n;
    // the end, to the loaders, both issuers and the three warpgroups
    ok = ok && hand_part(~0u);
    for (int i = 0; ok && i < kBufs; ++i, ++n) {
      ok = stage_free();
      if (!ok) break;
      if (lane == 0) {
        s.q_info[n % kStages] = kEnd;
        s.item[n % kStages] = make_uint4(kEnd, 0u, 0u, 0u);
        mbar_arrive(&s.q_full[n % kStages]);
      }
      __syncwarp();
    }
    if (!ok) {
      // the copies in flight land before the CTA exits
      uint32_t dummy_abort = 0;
      WaitCtl dw{nullptr, &dummy_abort, p.wait_ns};
      for (uint32_t i = loads > kStages ? loads - kStages : 0; i < loads; ++i)
        (void)mbar_wait(&s.q_full[i % kStages], (i / kStages) & 1u, dw);
    }
  } else if (warp < 3) {
    // ------------------------------------------------ MMA issuers (whole warps): items warp - 1, + 2, ...
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    constexpr uint64_t kTileDesc = kTileBytes >> 4;
    const uint64_t qdesc0 = sdesc_sw128(smem_u32(s.q[0]), 16, 1024);
    const uint64_t odesc = sdesc_plain(smem_u32(s.ones), 128, 256);
    const uint64_t tdesc0 = sdesc_plain(smem_u32(s.term[0]), 128, 256);
    for (uint32_t n = static_cast<uint32_t>(warp) - 1u;; n += 2) {
      const uint32_t st = n % kStages, b = n % kBufs;
      if (!mbar_wait_warp(&s.q_full[st], (n / kStages) & 1u, wc)) break;
      const uint32_t info = __shfl_sync(0xffffffffu, s.q_info[st], 0);
      if (info & kEnd) break;
      const uint32_t kb = info & 1u;
      if (!mbar_wait_warp(&s.k_full[kb], (info >> 8) & 1u, wc)) break;
      // The buffer's last item, n - 3, is the other issuer's.  Its scores are waited for first: without that this
      // warp could get here while the buffer still holds item n - 6, and take that item's phase of s_empty, two
      // phases back and of the same parity, for the one it needs.  (Item n - 6's scores are there: the producer
      // has seen its stage released before it loaded item n.)
      if (n >= static_cast<uint32_t>(kBufs) && (!mbar_wait_warp(&s.s_full[b], (n / kBufs - 1) & 1u, wc) ||
                                                !mbar_wait_warp(&s.s_empty[b], (n / kBufs - 1) & 1u, wc)))
        break;
      tc_fence_after();
      const uint64_t qd = qdesc0 + st * kTileDesc;
      const uint32_t d = BSA_TMEM(tmem + b * 128, 128u, p.err), ka = BSA_TMEM(tmem + kColK + kb * 64, D / 2u, p.err);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
        mma_ts_elect(d, ka + kk * 8, qd + off, idesc, kk > 0 ? 1u : 0u);
      }
      if constexpr (!kCap) mma_ss_elect(d, odesc, tdesc0 + st * (4096 >> 4), idesc, 1u);
      mma_commit_elect(&s.s_full[b]);
    }
    mma_commit_elect(&s.drain[warp - 1]);
    uint32_t dummy_abort = 0;
    WaitCtl dw{p.err, &dummy_abort, p.wait_ns};
    (void)mbar_wait(&s.drain[warp - 1], 0, dw);
  } else if (warp < kEwWarp0) {
    // ------------------------------------------------ K into tensor memory: a row per lane
    const int quarter = warp & 3;
    for (uint32_t k = 0;; ++k) {
      const uint32_t kb = k & 1u;
      if (!mbar_wait_warp(&s.part_full[kb], (k >> 1) & 1u, wc)) break;
      const uint32_t row = s.part_row[kb];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.part_read[kb]);
      if (row == ~0u) break;
      const int64_t r = BSA_RANGE(static_cast<int64_t>(row) + quarter * 32 + lane, int64_t(0),
                                  static_cast<int64_t>(p.B) * p.Hkv * p.Skv, p.err);
      const uint4* src = reinterpret_cast<const uint4*>(p.k + r * D);
      uint32_t v[D / 2];
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 q = __ldg(src + i);
        v[4 * i] = q.x;
        v[4 * i + 1] = q.y;
        v[4 * i + 2] = q.z;
        v[4 * i + 3] = q.w;
      }
      const uint32_t to = BSA_TMEM(tmem + kColK + kb * 64 + (static_cast<uint32_t>(quarter * 32) << 16), D / 2u, p.err);
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < D / 2; i += 32) tmem_st32(to + i, v + i);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.k_full[kb]);
    }
  } else {
    // ------------------------------------------------ exponentials: warpgroup w takes items w, w + 3, ...
    const int w = (warp - kEwWarp0) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;  // key of the tile == tensor-memory lane
    const uint32_t taddr = BSA_TMEM(tmem + w * 128 + (static_cast<uint32_t>(quarter * 32) << 16), 128u, p.err);
    const int32_t parts = c1.tile - c0.tile + (c1.skip > 0 ? 1 : 0);
    int32_t part = 0;
    uint64_t acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f2_pack(0.f, 0.f);
    // the finished parts' sums (zeros where this warpgroup had no item)
    auto flush_to = [&](int32_t to) {
      for (; part < to; ++part) {
        float a, b;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), a, b);
        p.sums[(static_cast<int64_t>(sums_row(p, blockIdx.x, c0.tile + part)) * kBufs + w) * 128 + r] = a + b;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = f2_pack(0.f, 0.f);
      }
    };
    for (uint32_t n = static_cast<uint32_t>(w);; n += kBufs) {
      const uint32_t st = n % kStages;
      if (!mbar_wait_warp(&s.q_full[st], (n / kStages) & 1u, wc)) break;
      const uint4 x = s.item[st];
      if (x.x & kEnd) {
        flush_to(parts);
        break;
      }
      flush_to(static_cast<int32_t>(x.z));
      const bool masked = x.x & kMask;
      Visible m{{~0u, ~0u, ~0u, ~0u}};
      if (masked) m = visible_queries(p, x, static_cast<int64_t>((c0.tile + part) % p.mi.rows) * 128 + r, r);
      if (!mbar_wait_warp(&s.s_full[w], (n / kBufs) & 1u, wc)) break;
      tc_fence_after();
      const float* term = reinterpret_cast<const float*>(s.term[st]);
      if constexpr (!kCap) {  // the scores are all that is left of the stage
        __syncwarp();
        mbar_arrive_cnt_elect(&s.stage_empty[st], 1u);
      }
      uint32_t va[32], vb[32];
      if (!masked) {
        // each load runs under the exponentials of the chunk before it (no branch while one is in flight)
        tmem_ld32(taddr, va);
        tmem_wait_ld();
        reg_fence32(va);
        tmem_ld32(taddr + 32, vb);
        add_probs<kCap>(p, va, term, acc);
        tmem_wait_ld();
        reg_fence32(vb);
        tmem_ld32(taddr + 64, va);
        add_probs<kCap>(p, vb, term + 32, acc);
        tmem_wait_ld();
        reg_fence32(va);
        tmem_ld32(taddr + 96, vb);
        add_probs<kCap>(p, va, term + 64, acc);
        tmem_wait_ld();
        reg_fence32(vb);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_cnt_elect(&s.s_empty[w], 1u);
        add_probs<kCap>(p, vb, term + 96, acc);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld32(taddr + 32 * c, va);
          tmem_wait_ld();
          reg_fence32(va);
          hide<kCap>(p, va, m.w[c]);
          add_probs<kCap>(p, va, term + 32 * c, acc);
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_cnt_elect(&s.s_empty[w], 1u);
      }
      if constexpr (kCap) {
        __syncwarp();
        mbar_arrive_cnt_elect(&s.stage_empty[st], 1u);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One block per tile: its rows of sums (three of each CTA that had a part of it) added up in order.
__global__ void __launch_bounds__(128) key_weights_join(const __grid_constant__ KwParams p) {
  griddep_wait();
  const int32_t t = static_cast<int32_t>(blockIdx.x);
  // the CTA whose run holds the tile's beginning: the last cut at or before it
  int32_t lo = 0, hi = p.n_cta;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) / 2;
    const Cut c = p.cut[mid];
    if (c.tile < t || (c.tile == t && c.skip == 0)) lo = mid;
    else hi = mid;
  }
  float v = 0.f;
  for (int32_t c = lo; c < p.n_cta && (c == lo || (p.cut[c].tile == t && p.cut[c].skip > 0)); ++c) {
    const float* row = p.sums + static_cast<int64_t>(sums_row(p, c, t)) * kBufs * 128 + threadIdx.x;
#pragma unroll
    for (int w = 0; w < kBufs; ++w) v += row[w * 128];
  }
  p.out[static_cast<int64_t>(t / p.mi.rows) * p.Skv + t % p.mi.rows * 128 + threadIdx.x] = v;
}

// The cuts: n_cta runs of equal cost in tile order.  A tile costs its items
// plus, for what its beginning and its masked items take, 2 + G more (measured
// on GQA 32/8 causal 8192: ~4,600 cycles a tile against ~765 an item; with
// items alone the CTAs that get the short tiles of a triangle end 18% after
// the others).  A cut inside that extra moves to the tile's beginning.
void make_cuts(const bsa_key_weights_args* a, const bsa_mask_info* info, KwParams* p) {
  const int32_t rows = info->rows, G = a->Hq / a->Hkv;
  const int32_t* len = info->row_len_h.data();
  // the tiles of one (b, g) (shared mask) or one b (per-head masks) repeat
  const int32_t per_tiles = info->heads == 1 ? rows : rows * a->Hkv;
  auto items = [&](int32_t t) -> int64_t {
    if (info->heads == 1) return static_cast<int64_t>(len[t]) * G;
    int64_t n = 0;
    for (int32_t i = 0; i < G; ++i) n += len[(t / rows * G + i) * rows + t % rows];
    return n;
  };
  const int64_t extra = 2 + G;
  auto cost = [&](int32_t t) -> int64_t {
    const int64_t n = items(t);
    return n > 0 ? n + extra : 0;
  };
  int64_t per = 0, per_items = 0;
  for (int32_t t = 0; t < per_tiles; ++t) {
    per += cost(t);
    per_items += items(t);
  }
  const int32_t periods = info->heads == 1 ? a->B * a->Hkv : a->B;
  const int64_t total = per * periods;
  p->n_cta = static_cast<int32_t>(
      std::max<int64_t>(1, std::min<int64_t>(per_items * periods, std::min(num_sms(), kMaxCtas))));
  p->cut[0] = Cut{0, 0};
  p->cut[p->n_cta] = Cut{per_tiles * periods, 0};
  int32_t t = 0;
  int64_t before = 0, period = 0;  // cost of the period's tiles before t
  for (int32_t c = 1; c < p->n_cta; ++c) {
    const int64_t at = total * c / p->n_cta;
    if (at / per != period) {
      period = at / per;
      t = 0;
      before = 0;
    }
    const int64_t rest = at - period * per;
    while (before + cost(t) <= rest) before += cost(t++);
    p->cut[c] = Cut{static_cast<int32_t>(period * per_tiles + t), static_cast<int32_t>(std::max<int64_t>(0, rest - before - extra))};
  }
}

template <int D, bool kCap>
bsa_status launch(const bsa_key_weights_args* a, const KwParams& p, cudaStream_t stream) {
  CUtensorMap tq;
  const int64_t q_rows = static_cast<int64_t>(a->B) * a->Hq * a->S_q;
  if (!make_tmap_bf16_panels(&tq, a->q, q_rows, D, 128))
    return fail(BSA_ERR_CUDA, "cuTensorMapEncodeTiled rejected the Q description");
  auto kern = key_weights_kernel<D, kCap>;
  const size_t smem = sizeof(KwSmem<D>) + 1024;
  const bsa_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem, "set key weights smem size");
  if (st != BSA_OK) return st;
  cudaError_t e = launch_kernel(key_weights_terms<kCap>, dim3(static_cast<unsigned>((q_rows + 255) / 256)), dim3(256), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "key weights terms launch");
  e = launch_kernel(kern, dim3(p.n_cta), dim3(kThreads), smem, stream, tq, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "key weights launch");
  e = launch_kernel(key_weights_join, dim3(p.n_tiles), dim3(128), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "key weights join launch");
  return BSA_OK;
}

// Floats of the rows of sums: one per warpgroup for each tile and each CTA's two shared parts.
size_t sums_floats(const bsa_key_weights_args* a, const bsa_mask_info* info) {
  return (static_cast<size_t>(a->B) * a->Hkv * info->rows + 2 * kMaxCtas) * kBufs * 128;
}

}  // namespace

size_t key_weights_workspace_bytes(const bsa_key_weights_args* a, const bsa_mask_info* info) {
  const size_t blocks = static_cast<size_t>(a->B) * a->Hq * (a->S_q / 128);
  return sums_floats(a, info) * sizeof(float) + blocks * (a->logits_soft_cap > 0.f ? Terms<true>::kBytes : Terms<false>::kBytes);
}

bsa_status key_weights_launch(const bsa_key_weights_args* a, const bsa_mask_info* info, float scale, cudaStream_t stream) {
  const size_t n = static_cast<size_t>(info->heads) * info->rows;
  if (info->row_len_h.size() < n) return fail(BSA_ERR_INVALID_ARG, "MaskInfo without its host row arrays");
  if (static_cast<int64_t>(a->B) * a->Hkv * info->rows > INT32_MAX - 1) return fail(BSA_ERR_UNSUPPORTED, "too many key blocks");
  KwParams p{};
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.Sq = a->S_q;
  p.Skv = a->S_kv;
  const bool cap = a->logits_soft_cap > 0.f;
  p.scale_log2 = cap ? scale / a->logits_soft_cap : scale * kLog2e;
  // (a scale of 0 would turn what hides a score into a NaN, and the terms are divided by it; products with
  // anything this small are as good as 0)
  if (std::fabs(p.scale_log2) < 1e-36f) p.scale_log2 = std::copysign(1e-36f, p.scale_log2);
  p.term_scale = cap ? -kLog2e : -kLog2e / p.scale_log2;
  p.hidden = cap ? -INFINITY : std::copysign(3e38f, -p.scale_log2);
  p.cap_log2 = a->logits_soft_cap > 0.f ? a->logits_soft_cap * kLog2e : 0.f;
  p.lse = a->lse;
  p.q_lens = a->q_lens;
  p.out = a->weights;
  p.sums = static_cast<float*>(a->workspace);
  p.n_tiles = a->B * a->Hkv * info->rows;
  p.terms = p.sums + sums_floats(a, info);
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.mi = mask_info_dev(info);
  p.compact = info->shrink ? 1 : 0;
  make_cuts(a, info, &p);
  p.err = device_error_word();
  p.wait_ns = wait_limit_ns();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  if (a->D == 128) return cap ? launch<128, true>(a, p, stream) : launch<128, false>(a, p, stream);
  return cap ? launch<64, true>(a, p, stream) : launch<64, false>(a, p, stream);
}

}  // namespace bsa
