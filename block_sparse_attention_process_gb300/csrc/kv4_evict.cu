// Eviction from the 4-bit cache by accumulated attention weight.
//
// Per (sequence, key head): the `keep` slots of the largest key, key = the
// weight as an ordered 32-bit integer (recent tokens above everything, NaN
// above every number), ties to the lower slot.  A radix select of three digits
// (11, 11 and 10 bits) finds the smallest kept key; every kept slot's place then follows
// from prefix counts, and a second kernel moves the rows.
//
// The selection reads 8 bytes a slot once and is otherwise latency: a cluster
// of up to 8 CTAs shares a head, each with its slice's keys in shared memory,
// and adds up its histograms through distributed shared memory.  One CTA a
// head that read the weights again for every digit took 193 us for 8 heads of
// 65,536 slots and 25 us for 128 heads of 1088; this takes 24 and 12 us
// (four digits of 8 bits: 26 and 14; the wider first one also spreads the
// atomics, as most weights share their exponent's top bits).  The
// move reads and writes D + D / 8 bytes a kept slot (and writes 4 D of values,
// if asked): 128 heads that keep 1024 of 1088 slots of 128 with their values,
// 106 MB, 22 us.
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kCachedKeys = 40 * 1024;  // keys of a slice kept in shared memory (160 KiB); a longer slice reads them again
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;  // of a digit (64 to each of 32 coarse ones)

struct EvictParams {
  bsa_kv4_cache c, o;
  const int32_t *lens, *seen;
  int64_t keep, recent;
  int32_t in_place;
  int32_t* new_lens;
  int32_t* index;
  __nv_bfloat16 *k_values, *v_values;
  int32_t* holes;  // workspace [B, Hkv, keep] (in place only)
  int32_t cluster;
  int32_t cached;  // keys a slice may keep in shared memory
  uint32_t* err;
};

// Weights as unsigned integers in increasing order.
__device__ __forceinline__ uint32_t order_key(float w, bool recent) {
  if (recent) return 0xFFFFFFFFu;
  if (isnan(w)) return 0xFFFFFFFEu;
  const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 and 0 are equal)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster; memory written before is visible after.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Two words of another CTA's shared memory.
__device__ __forceinline__ uint2 load_remote(const uint32_t* mine, uint32_t rank) {
  uint32_t a;
  uint2 v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Exclusive prefix sums over the CTA's threads of two counts, and their totals.
__device__ __forceinline__ void block_prefix(int32_t& a, int32_t& b, int32_t (*sums)[2], int32_t& all_a, int32_t& all_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int32_t ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int32_t xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += xa;
      ib += xb;
    }
  }
  if (lane == 31) {
    sums[warp][0] = ia;
    sums[warp][1] = ib;
  }
  __syncthreads();
  int32_t before_a = 0, before_b = 0;
  all_a = all_b = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w == warp) {
      before_a = all_a;
      before_b = all_b;
    }
    all_a += sums[w][0];
    all_b += sums[w][1];
  }
  a = before_a + ia - a;
  b = before_b + ib - b;
}

// One head per cluster; CTA r takes the r-th slice of its slots.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t keys[];  // the slice's, if it is short enough
  __shared__ __align__(8) uint32_t hist[2][kBins];  // (two: a CTA may still read one while the next digit's is counted)
  __shared__ __align__(8) uint32_t coarse[2][32];   // sums of kBins / 32 neighbouring bins
  __shared__ uint32_t pick[2];
  __shared__ __align__(8) uint32_t counts[4];  // slots of the slice above the least kept key, at it, and stays below slot keep
  __shared__ int32_t sums[kSelThreads / 32][2];
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t cta = cluster_rank(), C = static_cast<uint32_t>(p.cluster);
  const int64_t bh = blockIdx.x / C;
  const int32_t b = static_cast<int32_t>(bh / p.c.Hkv);
  const int32_t n = clamp_len(p.lens[b], p.c.capacity, threadIdx.x == 0 ? p.err : nullptr);
  const int64_t first_recent = static_cast<int64_t>(p.seen ? p.seen[b] : p.lens[b]) - p.recent;
  const float* w = p.c.weights + bh * p.c.capacity;
  const int32_t* pos = p.c.positions ? p.c.positions + bh * p.c.capacity : nullptr;
  int32_t* index = p.index + bh * p.keep;
  const int32_t keep = static_cast<int32_t>(p.keep < n ? p.keep : n);
  if (threadIdx.x == 0 && cta == 0 && bh % p.c.Hkv == 0) p.new_lens[b] = keep;
  const int32_t thread = static_cast<int32_t>(cta * kSelThreads + threadIdx.x), threads = static_cast<int32_t>(C * kSelThreads);
  for (int64_t r = keep + static_cast<int64_t>(thread); r < p.keep; r += threads) index[r] = -1;
  if (n <= p.keep) {  // (uniform over the cluster) everything stays
    for (int32_t i = thread; i < n; i += threads) index[i] = i;
    return;
  }
  // this CTA's slice, and this thread's run of it
  const int32_t chunk = (n + threads - 1) / threads | 1;  // (odd: a warp's runs start in different banks)
  const int32_t s0 = static_cast<int32_t>(min(static_cast<int64_t>(n), static_cast<int64_t>(cta) * kSelThreads * chunk));
  const int32_t s1 = static_cast<int32_t>(min(static_cast<int64_t>(n), static_cast<int64_t>(s0) + kSelThreads * chunk));
  const bool cached = s1 - s0 <= p.cached;
  auto make_key = [&](int32_t i) {
    const bool recent = p.recent > 0 && (pos ? static_cast<int64_t>(pos[i]) : i) >= first_recent;
    return order_key(w[i], recent);
  };
  auto key_of = [&](int32_t i) { return cached ? keys[i - s0] : make_key(i); };
  if (cached) {
#pragma unroll 4
    for (int32_t i = s0 + static_cast<int32_t>(threadIdx.x); i < s1; i += kSelThreads) keys[i - s0] = make_key(i);
  }

  uint32_t prefix = 0, mask = 0;
  uint32_t want = static_cast<uint32_t>(p.keep);  // rank (1-based, from the top) among keys with this prefix
  for (int d = 0; d < 3; ++d) {  // digits of 11, 11 and 10 bits
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
    const uint32_t digits = d == 2 ? 1023u : 2047u;
    uint32_t* h = hist[d & 1];
    for (int i = static_cast<int>(threadIdx.x); i < kBins; i += kSelThreads) h[i] = 0;
    __syncthreads();
    // (whole warps go round together, and count at once where all their slots have one digit, as weights of 0 do;
    // gathering all equal digits of a warp instead took 2 us more for 8 heads of 65,536 slots)
#pragma unroll 4
    for (int32_t i0 = s0; i0 < s1; i0 += kSelThreads) {
      const int32_t i = i0 + static_cast<int32_t>(threadIdx.x);
      const uint32_t k = i < s1 ? key_of(i) : 0u;
      const bool in = i < s1 && (k & mask) == prefix;
      if (!__any_sync(0xffffffffu, in)) continue;
      const uint32_t digit = in ? (k >> shift) & digits : kBins;
      int one;  // the whole warp has one digit
      (void)__match_all_sync(0xffffffffu, digit, &one);
      if (one) {
        if ((threadIdx.x & 31) == 0) atomicAdd(&h[digit], 32u);
      } else if (in) {
        atomicAdd(&h[digit], 1u);
      }
    }
    __syncthreads();
    {
      const uint32_t w = threadIdx.x / 32, l = threadIdx.x % 32;
      uint32_t v = h[w * (kBins / 32) + l] + h[w * (kBins / 32) + 32 + l];
      v = __reduce_add_sync(0xffffffffu, v);
      if (l == 0) coarse[d & 1][w] = v;
    }
    if (C > 1) cluster_barrier();
    else __syncthreads();
    if (threadIdx.x < 32) {
      // from the top: the coarse bin in which the count reaches `want`, then the bin within it
      const uint32_t lane = threadIdx.x;
      // two neighbouring counts of all CTAs (loads without branches between them: all on their way at once)
      auto totals = [&](const uint32_t* at) -> uint2 {
        if (C == 1) return *reinterpret_cast<const uint2*>(at);
        uint2 x[kMaxCluster];
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) x[c] = load_remote(at, min(c, C - 1));
        uint2 v = make_uint2(0u, 0u);
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c)
          if (c < C) {
            v.x += x[c].x;
            v.y += x[c].y;
          }
        return v;
      };
      uint32_t left = want;  // (the same in every lane)
      auto reach = [&](uint32_t n) -> uint32_t {  // the lane whose n, added to those before it, reaches `left`
        uint32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= static_cast<uint32_t>(o)) upto += x;
        }
        const uint32_t at = static_cast<uint32_t>(__ffs(__ballot_sync(0xffffffffu, upto >= left))) - 1u;
        left -= __shfl_sync(0xffffffffu, upto - n, at);
        return at;
      };
      const uint2 both = totals(&coarse[d & 1][(31u - lane) & ~1u]);
      const uint32_t top = 31u - reach(lane & 1 ? both.x : both.y);
      const uint32_t* bins = h + top * (kBins / 32);
      const uint2 two = totals(bins + 62u - 2u * lane);  // two neighbours a lane
      const uint32_t hi = two.y, lo = two.x;
      const uint32_t pair = reach(hi + lo);
      const uint32_t first = __shfl_sync(0xffffffffu, hi, pair);
      const bool second = left > first;
      if (second) left -= first;
      if (lane == 0) {
        pick[0] = top * (kBins / 32) + 63u - 2u * pair - (second ? 1u : 0u);
        pick[1] = left;
      }
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    mask |= digits << shift;
    want = pick[1];
    // (pick is written again only behind the next digit's barriers)
  }
  // `want` slots whose key is `prefix` stay, the lowest ones, and all above it

  const int32_t t0 = static_cast<int32_t>(min(static_cast<int64_t>(s1), s0 + static_cast<int64_t>(threadIdx.x) * chunk));
  const int32_t t1 = min(s1 - t0, chunk) + t0;
  int32_t above = 0, ties = 0;
  for (int32_t i = t0; i < t1; ++i) {
    const uint32_t k = key_of(i);
    above += k > prefix;
    ties += k == prefix;
  }
  int32_t all_above, all_ties;
  block_prefix(above, ties, sums, all_above, all_ties);
  if (threadIdx.x == 0) {
    counts[0] = static_cast<uint32_t>(all_above);
    counts[1] = static_cast<uint32_t>(all_ties);
    counts[2] = 0;
  }
  cluster_barrier();
  if (threadIdx.x < 32) {  // the CTAs before this one, a lane each
    const uint2 x = threadIdx.x < C ? load_remote(counts, threadIdx.x) : make_uint2(0u, 0u);
    const uint32_t a = __reduce_add_sync(0xffffffffu, threadIdx.x < cta ? x.x : 0u);
    const uint32_t t = __reduce_add_sync(0xffffffffu, threadIdx.x < cta ? x.y : 0u);
    if (threadIdx.x == 0) {
      pick[0] = a;
      pick[1] = t;
    }
  }
  __syncthreads();
  above += static_cast<int32_t>(pick[0]);
  ties += static_cast<int32_t>(pick[1]);
  const int32_t quota = static_cast<int32_t>(want);
  // stays before slot i: those above the least key, and ties up to the quota
  if (!p.in_place) {
    for (int32_t i = t0; i < t1; ++i) {
      const uint32_t k = key_of(i);
      const int32_t r = above + min(ties, quota);
      if (k > prefix || (k == prefix && ties < quota)) index[r] = i;
      above += k > prefix;
      ties += k == prefix;
    }
    cluster_barrier();  // (no CTA leaves while another reads its counts)
    return;
  }
  // in place: holes (slots below keep that are freed) by rank, then the stays from slot keep on into them
  int32_t a = above, t = ties;
  for (int32_t i = t0; i < t1; ++i) {
    const uint32_t k = key_of(i);
    const int32_t stays = a + min(t, quota);
    if (i == keep) counts[2] = static_cast<uint32_t>(stays);  // (one thread of the cluster)
    if (i < keep) {
      if (k > prefix || (k == prefix && t < quota)) index[i] = i;
      else p.holes[bh * p.keep + i - stays] = i;
    }
    a += k > prefix;
    t += k == prefix;
  }
  cluster_barrier();  // the holes are written (and n > keep: slot keep has been met)
  if (threadIdx.x < 32) {
    const uint32_t n = __reduce_add_sync(0xffffffffu, threadIdx.x < C ? load_remote(counts + 2, threadIdx.x).x : 0u);
    if (threadIdx.x == 0) pick[0] = n;
  }
  __syncthreads();
  const uint32_t below = pick[0];
  a = above;
  t = ties;
  for (int32_t i = t0; i < t1; ++i) {
    const uint32_t k = key_of(i);
    const int32_t stays = a + min(t, quota);
    if (i >= keep && (k > prefix || (k == prefix && t < quota)))
      index[p.holes[bh * p.keep + stays - static_cast<int32_t>(below)]] = i;
    a += k > prefix;
    t += k == prefix;
  }
  cluster_barrier();  // (no CTA leaves while another reads its counts)
}

// What the nibbles at bits 0-3 and 16-19 of x stand for, as bf16: 128 + c is
// exact in bf16, so is (128 + c) - 136, and the product is rounded once.
__device__ __forceinline__ uint32_t code_values(uint32_t x, uint32_t scale2) {
  uint32_t y, z;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"((x & 0x000F000Fu) | 0x43004300u), "r"(0x43084308u));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(y), "r"(scale2));
  return z;
}
// The eight elements of a word in order, under the scales (bf16 bits) of its
// low and high four.
__device__ __forceinline__ uint4 word_values(uint32_t w, uint32_t s_lo, uint32_t s_hi) {
  const uint32_t s = __byte_perm(s_lo, s_hi, 0x5410);  // nibbles i and i + 4 go together
  const uint32_t a = code_values(w, s), b = code_values(w >> 4, s), c = code_values(w >> 8, s), d = code_values(w >> 12, s);
  return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632), __byte_perm(c, d, 0x7632));
}

constexpr int kMoves = 2;  // rows of one head that a lane has in flight

template <int D>
__global__ void __launch_bounds__(256) move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kLanes = Kv4<D>::kWords;
  constexpr int kPiece = Kv4<D>::kPieceWords;
  constexpr int kGroups = Kv4<D>::kGroups;
  constexpr int kRowsCta = 256 / kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const int u = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int64_t heads = static_cast<int64_t>(p.c.B) * p.c.Hkv;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRowsCta;
  for (int64_t bh = blockIdx.y; bh < heads; bh += gridDim.y)
    for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRowsCta + sub; r0 < p.keep; r0 += step * kMoves) {
      int32_t src[kMoves];
      uint32_t kw[kMoves], vw[kMoves], ks[kMoves], vs[kMoves];
#pragma unroll
      for (int i = 0; i < kMoves; ++i) src[i] = r0 + i * step < p.keep ? p.index[bh * p.keep + r0 + i * step] : -1;
#pragma unroll
      for (int i = 0; i < kMoves; ++i) {
        kw[i] = vw[i] = 0x88888888u;
        ks[i] = vs[i] = 0;
        if (src[i] < 0) continue;
        const int64_t from = bh * p.c.capacity + src[i];
        kw[i] = static_cast<const uint32_t*>(p.c.k_codes)[from * kLanes + u];
        vw[i] = static_cast<const uint32_t*>(p.c.v_codes)[from * kLanes + (u ^ v_word_swap<D>(src[i]))];
        ks[i] = static_cast<const uint16_t*>(p.c.k_scales)[from * kGroups + u % kGroups];
        vs[i] = static_cast<const uint32_t*>(p.c.v_scales)[from * kPiece + u % kPiece];
      }
#pragma unroll
      for (int i = 0; i < kMoves; ++i) {
        const int64_t r = r0 + i * step;
        if (r >= p.keep) continue;
        if (src[i] >= 0 && !(p.in_place && src[i] == r)) {
          const int64_t from = bh * p.c.capacity + src[i], to = bh * p.o.capacity + r;
          static_cast<uint32_t*>(p.o.k_codes)[to * kLanes + u] = kw[i];
          static_cast<uint32_t*>(p.o.v_codes)[to * kLanes + (u ^ v_word_swap<D>(r))] = vw[i];
          if (u < kGroups) static_cast<uint16_t*>(p.o.k_scales)[to * kGroups + u] = static_cast<uint16_t>(ks[i]);
          if (u < kPiece) static_cast<uint32_t*>(p.o.v_scales)[to * kPiece + u] = vs[i];
          if (u == 0 && p.o.weights) p.o.weights[to] = p.c.weights[from];
          if (u == 1 && p.o.positions) p.o.positions[to] = p.c.positions ? p.c.positions[from] : src[i];
        }
        const int64_t row = (bh * p.keep + r) * D;
        if (p.k_values) __stcs(reinterpret_cast<uint4*>(p.k_values + row + k_word_elem<D>(u)), word_values(kw[i], ks[i], ks[i]));
        if (p.v_values) {
          const uint4 o = word_values(vw[i], vs[i] & 0xFFFFu, vs[i] >> 16);
          __stcs(reinterpret_cast<uint2*>(p.v_values + row + v_word_elem<D>(u, 0)), make_uint2(o.x, o.y));
          __stcs(reinterpret_cast<uint2*>(p.v_values + row + v_word_elem<D>(u, 1)), make_uint2(o.z, o.w));
        }
      }
    }
}

}  // namespace

size_t kv4_evict_workspace_bytes(const bsa_kv4_evict_args* a) {
  const bool in_place = a->out.k_codes == a->cache.k_codes;
  return in_place ? static_cast<size_t>(a->cache.B) * a->cache.Hkv * a->keep * sizeof(int32_t) : 0;
}

bsa_status kv4_evict_launch(const bsa_kv4_evict_args* a, cudaStream_t stream) {
  EvictParams p{};
  p.c = a->cache;
  p.o = a->out;
  p.lens = a->lens;
  p.seen = a->seen;
  p.keep = a->keep;
  p.recent = a->recent;
  p.in_place = a->out.k_codes == a->cache.k_codes;
  p.new_lens = a->new_lens;
  p.index = a->index;
  p.k_values = static_cast<__nv_bfloat16*>(a->k_values);
  p.v_values = static_cast<__nv_bfloat16*>(a->v_values);
  p.holes = static_cast<int32_t*>(a->workspace);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  // CTAs a head: more while SMs are free and a slice has 2048 slots or more
  const int64_t heads = static_cast<int64_t>(a->cache.B) * a->cache.Hkv;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && heads * p.cluster * 2 <= num_sms() && a->cache.capacity / p.cluster >= 4096) p.cluster *= 2;
  const int64_t slice = ((a->cache.capacity + p.cluster * kSelThreads - 1) / (p.cluster * kSelThreads) | 1) * kSelThreads;
  p.cached = slice <= kCachedKeys ? static_cast<int32_t>(slice) : 0;
  const size_t smem = static_cast<size_t>(p.cached) * sizeof(uint32_t);
  const bsa_status st = ensure_smem_attr(reinterpret_cast<const void*>(select_kernel), kCachedKeys * sizeof(uint32_t), "set selection smem size");
  if (st != BSA_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(heads * p.cluster));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 evict selection launch");
  const int64_t per = 256 / (a->cache.D / 8) * kMoves;
  const unsigned gy = static_cast<unsigned>(std::min<int64_t>(heads, 65535));
  const unsigned gx = static_cast<unsigned>(std::min<int64_t>((a->keep + per - 1) / per, std::max<int64_t>(1, num_sms() * 16 / gy)));
  e = a->cache.D == 128 ? launch_kernel(move_kernel<128>, dim3(gx, gy), dim3(256), 0, stream, p)
                        : launch_kernel(move_kernel<64>, dim3(gx, gy), dim3(256), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 evict move launch");
  return BSA_OK;
}

}  // namespace bsa
