// The attention weight every key of a prompt has received:
//   w[j] = sum over the group's q heads and the queries i that see j of exp(scale q_i.k_j - lse_i).
// The loop is the dK/dV launch's: a tile is a key block of one key head, its
// items the non-empty query blocks of each q head's row of the dkv MaskInfo.
//
// Per item one 128 x 128 x D product and 128^2 exponentials.  Queries are the
// product's M side (tensor-memory lanes), keys its columns: a row's logsumexp
// is then one register of a thread, and the sum over the queries stays in 32
// registers per thread (one per key column) until the tile ends, when the
// lanes are summed once.
//
// One persistent CTA per SM, warp-specialised:
//   warp 0      walks MaskInfo; loads K per tile (2 buffers), Q per item (4
//               stages) and its logsumexp, and publishes the items and the
//               ends of tiles in a ring
//   warp 1      tcgen05 issuer: S = Q K^T into one of four tensor-memory buffers
//   warp 2      adds up the warps' column sums at a tile's end and writes them
//   warps 4-19  exponentials: warp (part, quarter) takes 32 lanes x 32 columns
// All items of the launch form one sequence, cut into equal runs, one per CTA
// (the host computes the cuts from MaskInfo's row lengths and passes them as
// kernel parameters: no schedule to upload).  A tile that two or more CTAs
// share leaves one partial row per CTA in the workspace, and a second kernel
// adds these up in CTA order.
#include <cmath>

#include "internal.h"
#include "maskinfo_dev.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace bsa {
namespace {

constexpr int kBufs = 4;        // Q stages and score buffers (an item's have the same index)
constexpr int kRing = 8;        // entries (items and tile ends) between the walker and the others
constexpr int kParts = 4;       // warpgroups of the exponentials, 32 columns each
constexpr int kEwWarps = 4 * kParts;
constexpr int kThreads = 128 + 32 * kEwWarps;
constexpr uint32_t kRingReaders = 2 + kEwWarps;
constexpr int kMaxCtas = 160;
constexpr float kLog2e = 1.4426950408889634f;

// flags of an entry, beside its column (bits 0-15) and label (16-17)
constexpr uint32_t kFirst = 1u << 20;    // first item of its part of a tile
constexpr uint32_t kMask = 1u << 21;     // some pairs of the item are not visible
constexpr uint32_t kTileEnd = 1u << 22;  // end of a part: y = output row, z = the part had items, w = partial slot + 1 or 0
constexpr uint32_t kEnd = 1u << 23;

template <int D>
struct __align__(1024) KwSmem {
  static constexpr int kTileBytes = 128 * D * 2;
  uint8_t k[2][kTileBytes];
  uint8_t q[kBufs][kTileBytes];
  float lse[kRing][128];
  float red[2][4][128];  // [tile parity][quarter][key]
  uint4 entry[kRing];
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t q_full[kBufs], s_full[kBufs], s_empty[kBufs];  // s_full also frees the Q stage
  uint64_t k_full[2], k_empty[2];
  uint64_t red_full[2], red_empty[2];
  uint64_t drain;
  uint32_t tmem_base, abort_flag;
};
static_assert(sizeof(KwSmem<128>) + 1024 <= 232448, "key weights shared memory exceeds 227 KB per CTA");

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
  float* out;
  float* partial;  // [n_cta][2][128]
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

template <int D, bool kCap>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ KwParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = KwSmem<D>;
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr uint32_t kTileBytes = Smem::kTileBytes;
  constexpr int kChunks = D / 64;
  const int warp = warp_id(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&s.ring_full[i], 1);
      mbar_init(&s.ring_empty[i], kRingReaders);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&s.q_full[i], 1);
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.s_empty[i], kEwWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.k_full[i], 1);
      mbar_init(&s.k_empty[i], 1);
      mbar_init(&s.red_full[i], kEwWarps);
      mbar_init(&s.red_empty[i], 1);
    }
    mbar_init(&s.drain, 1);
    fence_mbar_init();
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
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------ walker and producer
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      const uint64_t pol = policy_evict_last();
      uint32_t e = 0, n = 0, k_loads = 0, lse_pending = 0;
      bool ok = true;
      auto slot_free = [&]() -> bool {
        return e < static_cast<uint32_t>(kRing) || mbar_wait(&s.ring_empty[e % kRing], (e / kRing - 1) & 1u, wc);
      };
      const Cut c0 = p.cut[blockIdx.x], c1 = p.cut[blockIdx.x + 1];
      const int32_t G = p.Hq / p.Hkv;
      for (int32_t tile = c0.tile; ok && tile <= c1.tile; ++tile) {
        if (tile == c1.tile && c1.skip == 0) break;
        const int32_t j = tile % p.mi.rows, bg = tile / p.mi.rows, b = bg / p.Hkv, g = bg % p.Hkv;
        const int32_t all = tile_items(p, tile);
        const int32_t begin = tile == c0.tile ? c0.skip : 0;
        const int32_t stop = tile == c1.tile ? c1.skip : all;
        const int32_t q_end = query_end(p, b);
        const int64_t krow = static_cast<int64_t>(bg) * p.Skv + static_cast<int64_t>(j) * 128;
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
          const int32_t end = min(at + len, stop);
          int32_t pos = p.compact && at < begin ? begin - at : 0;
          at += pos;
          RawRef ahead = pos < p.mi.width ? load_block(p.mi, row_base, pos) : RawRef{0, 0, 0};
          for (; ok && at < end && pos < p.mi.width; ++pos) {
            const RawRef cur = ahead;
            if (pos + 1 < p.mi.width) ahead = load_block(p.mi, row_base, pos + 1);
            const BlockRef br = check_block(p.mi, cur, p.err);
            if (br.label == 0) continue;
            if (at++ < begin) continue;
            if (br.col * 128 >= q_end) continue;  // padding only
            const uint32_t st = n % kBufs;
            if (!slot_free()) { ok = false; break; }
            // the stage's last scores are computed: its Q has been read
            if (n >= static_cast<uint32_t>(kBufs) && !mbar_wait(&s.s_full[st], (n / kBufs - 1) & 1u, wc)) { ok = false; break; }
            const int64_t qrow = BSA_RANGE((static_cast<int64_t>(b) * p.Hq + hq) * p.Sq + static_cast<int64_t>(br.col) * 128,
                                           int64_t(0), static_cast<int64_t>(p.B) * p.Hq * p.Sq - 127, p.err);
            const bool mask = br.label == 1 || br.col * 128 + 128 > q_end;
            s.entry[e % kRing] = make_uint4(static_cast<uint32_t>(br.col) | static_cast<uint32_t>(br.label) << 16 |
                                                (first ? kFirst : 0u) | (mask ? kMask : 0u),
                                            static_cast<uint32_t>(br.slot), static_cast<uint32_t>(j),
                                            static_cast<uint32_t>(q_end));
            mbar_arrive_expect_tx(&s.ring_full[e % kRing], 512);
            bulk_load(s.lse[e % kRing], p.lse + qrow, 512, &s.ring_full[e % kRing]);
            lse_pending |= 1u << (e % kRing);
            ++e;
            mbar_arrive_expect_tx(&s.q_full[st], kTileBytes);
            for (int c = 0; c < kChunks; ++c)
              tma_load_2d(s.q[st] + c * 16384, &tm_q, &s.q_full[st], c * 64, static_cast<int32_t>(qrow), pol);
            ++n;
            if (first) {
              const uint32_t kb = k_loads & 1u;
              if (k_loads >= 2 && !mbar_wait(&s.k_empty[kb], (k_loads / 2 - 1) & 1u, wc)) { ok = false; break; }
              mbar_arrive_expect_tx(&s.k_full[kb], kTileBytes);
              for (int c = 0; c < kChunks; ++c)
                tma_load_2d(s.k[kb] + c * 16384, &tm_k, &s.k_full[kb], c * 64, static_cast<int32_t>(krow), pol);
              ++k_loads;
              first = false;
            }
          }
          at = end;
        }
        if (!ok || !slot_free()) { ok = false; break; }
        const bool whole = begin == 0 && stop == all;
        const uint32_t part = static_cast<uint32_t>(2 * blockIdx.x + (tile == c0.tile ? 0 : 1));
        s.entry[e % kRing] = make_uint4(kTileEnd, static_cast<uint32_t>(krow), first ? 0u : 1u, whole ? 0u : part + 1u);
        mbar_arrive(&s.ring_full[e % kRing]);
        lse_pending &= ~(1u << (e % kRing));
        ++e;
      }
      if (ok && slot_free()) {
        s.entry[e % kRing] = make_uint4(kEnd, 0u, 0u, 0u);
        mbar_arrive(&s.ring_full[e % kRing]);
        ++e;
      } else {
        // the copies in flight land before the CTA exits
        uint32_t dummy_abort = 0;
        WaitCtl dw{nullptr, &dummy_abort, p.wait_ns};
        for (uint32_t i = n > kBufs ? n - kBufs : 0; i < n; ++i) (void)mbar_wait(&s.q_full[i % kBufs], (i / kBufs) & 1u, dw);
        for (uint32_t i = k_loads > 2 ? k_loads - 2 : 0; i < k_loads; ++i) (void)mbar_wait(&s.k_full[i & 1u], (i / 2) & 1u, dw);
        for (uint32_t i = e > kRing ? e - kRing : 0; i < e; ++i)
          if (lse_pending >> (i % kRing) & 1u) (void)mbar_wait(&s.ring_full[i % kRing], (i / kRing) & 1u, dw);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer (whole warp)
    constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
    constexpr uint64_t kTileDesc = kTileBytes >> 4;
    const uint64_t qdesc0 = sdesc_sw128(smem_u32(s.q[0]), 16, 1024);
    const uint64_t kdesc0 = sdesc_sw128(smem_u32(s.k[0]), 16, 1024);
    uint32_t n = 0, k_uses = 0;
    for (uint32_t e = 0;; ++e) {
      const uint32_t slot = e % kRing;
      if (!mbar_wait_warp(&s.ring_full[slot], (e / kRing) & 1u, wc)) break;
      const uint4 x = s.entry[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.ring_empty[slot]);
      if (x.x & kEnd) break;
      if (x.x & kTileEnd) {
        if (x.z) {
          mma_commit_elect(&s.k_empty[k_uses & 1u]);
          ++k_uses;
        }
        continue;
      }
      if ((x.x & kFirst) && !mbar_wait_warp(&s.k_full[k_uses & 1u], (k_uses / 2) & 1u, wc)) break;
      const uint32_t b = n % kBufs;
      if (n >= static_cast<uint32_t>(kBufs) && !mbar_wait_warp(&s.s_empty[b], (n / kBufs - 1) & 1u, wc)) break;
      if (!mbar_wait_warp(&s.q_full[b], (n / kBufs) & 1u, wc)) break;
      tc_fence_after();
      const uint64_t qd = qdesc0 + b * kTileDesc, kd = kdesc0 + (k_uses & 1u) * kTileDesc;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>(((kk >> 2) * 16384 + (kk & 3) * 32) >> 4);
        mma_ss_elect(BSA_TMEM(tmem + b * 128, 128u, p.err), qd + off, kd + off, idesc, kk > 0 ? 1u : 0u);
      }
      mma_commit_elect(&s.s_full[b]);
      ++n;
    }
    mma_commit_elect(&s.drain);
    uint32_t dummy_abort = 0;
    WaitCtl dw{p.err, &dummy_abort, p.wait_ns};
    (void)mbar_wait(&s.drain, 0, dw);
  } else if (warp == 2) {
    // ------------------------------------------------ column sums of finished tiles
    uint32_t t = 0;
    for (uint32_t e = 0;; ++e) {
      const uint32_t slot = e % kRing;
      if (!mbar_wait_warp(&s.ring_full[slot], (e / kRing) & 1u, wc)) break;
      const uint4 x = s.entry[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.ring_empty[slot]);
      if (x.x & kEnd) break;
      if (!(x.x & kTileEnd)) continue;
      const uint32_t tp = t & 1u;
      if (!mbar_wait_warp(&s.red_full[tp], (t / 2) & 1u, wc)) break;
      float4 v = *reinterpret_cast<const float4*>(&s.red[tp][0][4 * lane]);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const float4 y = *reinterpret_cast<const float4*>(&s.red[tp][i][4 * lane]);
        v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.red_empty[tp]);
      const int64_t row = BSA_RANGE(static_cast<int64_t>(x.y), int64_t(0), static_cast<int64_t>(p.B) * p.Hkv * p.Skv - 127, p.err);
      float* dst = x.w ? p.partial + static_cast<int64_t>(x.w - 1) * 128 : p.out + row;
      *reinterpret_cast<float4*>(dst + 4 * lane) = v;
      ++t;
    }
  } else if (warp >= 4) {
    // ------------------------------------------------ exponentials
    const int part = (warp - 4) >> 2, quarter = (warp - 4) & 3;
    const int r = quarter * 32 + lane;  // query row of the item == tensor-memory lane
    const uint32_t taddr = tmem + part * 32 + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t sc2 = f2_pack(p.scale_log2, p.scale_log2);
    uint64_t acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = f2_pack(0.f, 0.f);
    uint32_t n = 0, t = 0;
    for (uint32_t e = 0;; ++e) {
      const uint32_t slot = e % kRing;
      if (!mbar_wait_warp(&s.ring_full[slot], (e / kRing) & 1u, wc)) break;
      const uint4 x = s.entry[slot];
      if (x.x & kEnd) break;
      if (x.x & kTileEnd) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.ring_empty[slot]);
        const uint32_t tp = t & 1u;
        if (t >= 2 && !mbar_wait_warp(&s.red_empty[tp], (t / 2 - 1) & 1u, wc)) break;
        // sum over the 32 lanes, column c ending in lane c: halves are exchanged
        float v[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          f2_unpack(acc[i], v[2 * i], v[2 * i + 1]);
          acc[i] = f2_pack(0.f, 0.f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        s.red[tp][quarter][part * 32 + lane] = v[0];
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.red_full[tp]);
        ++t;
        continue;
      }
      const float l = s.lse[slot][r];
      const float nl = l == -INFINITY ? -INFINITY : -l * kLog2e;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.ring_empty[slot]);
      uint32_t seen = 0xFFFFFFFFu;  // visible columns of this row
      if (x.x & kMask) {
        const int32_t col = static_cast<int32_t>(x.x & 0xFFFFu);
        const int64_t q = static_cast<int64_t>(col) * 128 + r;
        if (((x.x >> 16) & 3u) == 1u) {
          if (p.mi.kind == BSA_MASK_DENSE) {
            // word c of the block's rows (keys) part * 32 + c, bit = this query: loaded a row per lane, turned by shuffles
            const uint32_t word = __ldg(p.mi.partial_bits + (static_cast<int64_t>(x.y) * 128 + part * 32 + lane) * 4 + quarter);
            seen = 0;
#pragma unroll
            for (int c = 0; c < 32; ++c) seen |= ((__shfl_sync(0xffffffffu, word, c) >> lane) & 1u) << c;
          } else {
            int64_t lo, hi;
            key_interval(p.mi.kind, p.mi.left, p.mi.right, p.mi.chunk, q, lo, hi);
            const int64_t k0 = static_cast<int64_t>(x.z) * 128 + part * 32;
            const int64_t a = lo > k0 ? lo - k0 : 0, b = hi < k0 + 31 ? hi - k0 : 31;
            seen = b < a ? 0u : static_cast<uint32_t>((0xFFFFFFFFull >> (31 - (b - a))) << a);
          }
        }
        if (q >= static_cast<int64_t>(x.w)) seen = 0;
      }
      const uint32_t b = n % kBufs;
      if (!mbar_wait_warp(&s.s_full[b], (n / kBufs) & 1u, wc)) break;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(BSA_TMEM(taddr + b * 128, 32u, p.err), v);
      tmem_wait_ld();
      reg_fence32(v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.s_empty[b]);
      ++n;
      const uint64_t nl2 = f2_pack(nl, nl);
      if (!(x.x & kMask)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float e0, e1;
          if constexpr (kCap) {
            e0 = fmaf(tanh_fast(__uint_as_float(v[2 * i]) * p.scale_log2), p.cap_log2, nl);
            e1 = fmaf(tanh_fast(__uint_as_float(v[2 * i + 1]) * p.scale_log2), p.cap_log2, nl);
          } else {
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2, nl2), e0, e1);
          }
          acc[i] = f2_add(acc[i], f2_pack(ex2_approx(e0), ex2_approx(e1)));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float e0, e1;
          if constexpr (kCap) {
            e0 = fmaf(tanh_fast(__uint_as_float(v[2 * i]) * p.scale_log2), p.cap_log2, nl);
            e1 = fmaf(tanh_fast(__uint_as_float(v[2 * i + 1]) * p.scale_log2), p.cap_log2, nl);
          } else {
            f2_unpack(f2_fma(f2_pack(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), sc2, nl2), e0, e1);
          }
          const float p0 = (seen >> (2 * i)) & 1u ? ex2_approx(e0) : 0.f;
          const float p1 = (seen >> (2 * i + 1)) & 1u ? ex2_approx(e1) : 0.f;
          acc[i] = f2_add(acc[i], f2_pack(p0, p1));
        }
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

// Sums the partial rows of the tile that CTA c's run ends in (if it began
// there, or its run is the tile's first): those of c and the CTAs after it
// that have items of the same tile.
__global__ void __launch_bounds__(128) key_weights_join(const __grid_constant__ KwParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int32_t c = static_cast<int32_t>(blockIdx.x);
  const Cut mine = p.cut[c], next = p.cut[c + 1];
  if (next.skip == 0 || (mine.tile == next.tile && mine.skip > 0)) return;
  float v = p.partial[(2 * c + (mine.tile == next.tile ? 0 : 1)) * 128 + threadIdx.x];
  for (int32_t i = c + 1; i < p.n_cta && p.cut[i].tile == next.tile; ++i)
    if (p.cut[i].skip > 0) v += p.partial[2 * i * 128 + threadIdx.x];
  const int32_t bg = next.tile / p.mi.rows, j = next.tile % p.mi.rows;
  p.out[static_cast<int64_t>(bg) * p.Skv + j * 128 + threadIdx.x] = v;
}

// The cuts: n_cta equal runs of the items in tile order.
void make_cuts(const bsa_key_weights_args* a, const bsa_mask_info* info, KwParams* p) {
  const int32_t rows = info->rows, G = a->Hq / a->Hkv;
  const int32_t* len = info->row_len_h.data();
  // items of the tiles of one (b, g) (shared mask) or one b (per-head masks)
  const int32_t per_tiles = info->heads == 1 ? rows : rows * a->Hkv;
  auto items = [&](int32_t t) -> int64_t {
    if (info->heads == 1) return static_cast<int64_t>(len[t]) * G;
    int64_t n = 0;
    for (int32_t i = 0; i < G; ++i) n += len[(t / rows * G + i) * rows + t % rows];
    return n;
  };
  int64_t per = 0;
  for (int32_t t = 0; t < per_tiles; ++t) per += items(t);
  const int32_t periods = info->heads == 1 ? a->B * a->Hkv : a->B;
  const int64_t total = per * periods;
  p->n_cta = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(total, std::min(num_sms(), kMaxCtas))));
  p->cut[0] = Cut{0, 0};
  p->cut[p->n_cta] = Cut{per_tiles * periods, 0};
  // one pass over a period per group of cuts that fall into it
  int32_t t = 0;
  int64_t before = 0, period = 0;  // items of the period's tiles before t
  for (int32_t c = 1; c < p->n_cta; ++c) {
    const int64_t at = total * c / p->n_cta;
    if (at / per != period) {
      period = at / per;
      t = 0;
      before = 0;
    }
    const int64_t rest = at - period * per;
    while (before + items(t) <= rest) before += items(t++);
    p->cut[c] = Cut{static_cast<int32_t>(period * per_tiles + t), static_cast<int32_t>(rest - before)};
  }
}

template <int D>
bsa_status launch(const bsa_key_weights_args* a, const KwParams& p, cudaStream_t stream) {
  CUtensorMap tq, tk;
  if (!make_tmap_bf16_2d(&tq, a->q, static_cast<uint64_t>(a->B) * a->Hq * a->S_q, D, D * 2, 128, 64) ||
      !make_tmap_bf16_2d(&tk, a->k, static_cast<uint64_t>(a->B) * a->Hkv * a->S_kv, D, D * 2, 128, 64))
    return fail(BSA_ERR_CUDA, "cuTensorMapEncodeTiled rejected a Q/K description");
  auto kern = p.cap_log2 > 0.f ? key_weights_kernel<D, true> : key_weights_kernel<D, false>;
  const size_t smem = sizeof(KwSmem<D>) + 1024;
  const bsa_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem, "set key weights smem size");
  if (st != BSA_OK) return st;
  cudaError_t e = launch_kernel(kern, dim3(p.n_cta), dim3(kThreads), smem, stream, tq, tk, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "key weights launch");
  if (p.n_cta > 1) {
    e = launch_kernel(key_weights_join, dim3(p.n_cta), dim3(128), 0, stream, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "key weights join launch");
  }
  return BSA_OK;
}

}  // namespace

size_t key_weights_workspace_bytes(const bsa_key_weights_args*, const bsa_mask_info*) {
  return static_cast<size_t>(kMaxCtas) * 2 * 128 * sizeof(float);
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
  p.scale_log2 = a->logits_soft_cap > 0.f ? scale / a->logits_soft_cap : scale * kLog2e;
  p.cap_log2 = a->logits_soft_cap > 0.f ? a->logits_soft_cap * kLog2e : 0.f;
  p.lse = a->lse;
  p.q_lens = a->q_lens;
  p.out = a->weights;
  p.partial = static_cast<float*>(a->workspace);
  p.mi = mask_info_dev(info);
  p.compact = info->shrink ? 1 : 0;
  make_cuts(a, info, &p);
  p.err = device_error_word();
  p.wait_ns = wait_limit_ns();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  return a->D == 128 ? launch<128>(a, p, stream) : launch<64>(a, p, stream);
}

}  // namespace bsa
