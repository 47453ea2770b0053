// The pages worth attending to, for each query: those with the largest bound on q.k, q rounded to 8 bits.
//
// A page's keys lie between its bounds, so sum_d max(q_d hi_d, q_d lo_d) bounds q.k over the page.  With q+ =
// max(q, 0) and q- = min(q, 0) that is q+ hi + q- lo: one matrix product of length 2 D, [q+ | q-] [hi | lo]^T.
//
// Exactness.  q is taken as whole numbers of up to 8 bits (|qc| <= 128, times 2^f), the bounds are whole numbers
// |c| <= 256 times 2^e of the page.  Products are at most 2^15, their sums over D <= 128 channels (of a channel's two products
// one is 0) at most 2^22: multiples of 2^e that fp32 accumulators hold exactly, whatever the order.  2^f is the same for all of a
// query's pages and is left out.  So the choice is one and the same for every way to split the work, and ties are real ties.
//
// One launch, a cluster a query.  A warp scores 8 pages at a time as the narrow side of m16n8k16 products, the group's q
// heads being the 16-row side.  The channels of a product's k axis are taken in an order that makes a thread's share of 8
// pages 16-byte loads straight from memory (thread t of a quad: channels 8 t .. 8 t + 7 of every 32), the four of a
// quad 64 bytes side by side; nothing goes through shared memory but q.  The CTAs of the cluster take the pages in turn and write
// the scores, as ordered 32-bit keys, to the first one's shared memory.  That one chooses: keys less the smallest; counts of
// their digits, from the highest one on, give the least key that is kept and how many pages of it; then the
// kept pages in order, by prefix sums.
//
// 128 queries of 64 to 512 pages take 12 us (19 MB of bounds), 8 of 2048 11: some 5 until the first pages are scored, 3 for the
// choice; what bounds it is the latency of a chain of loads and barriers.
#include <algorithm>

#include "paged.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPassPages = kWarps * 8;  // pages that a CTA scores side by side
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kMaxPages = 49152;        // keys that the first CTA's shared memory holds
constexpr int kHeld = 8;  // keys a thread keeps in registers

struct SelectParams {
  const __nv_bfloat16* bounds;
  const __nv_bfloat16* q;
  int64_t qs[3];
  const int32_t *table, *lens, *q_lens;
  int32_t* index;
  int32_t B, Hkv, G, T, shift, pages;
  int64_t M;
  int32_t keep, first, recent;
  int32_t cluster;
  uint32_t* err;
};

// Pages that token t of sequence b sees (0: padding).
__device__ __forceinline__ int32_t pages_seen(const SelectParams& p, int32_t b, int32_t t, uint32_t* err) {
  const int32_t len = paged_len(p.lens[b], p.M << p.shift, err);
  const int32_t nq = p.q_lens ? paged_len(p.q_lens[b], p.T, err) : p.T;
  if (t >= nq) return 0;
  const int64_t end = static_cast<int64_t>(len) - nq + t + 1;  // keys
  return end <= 0 ? 0 : static_cast<int32_t>((end + (1 << p.shift) - 1) >> p.shift);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Order of scores as order of unsigned numbers.
__device__ __forceinline__ uint32_t ordered(float s) {
  const uint32_t x = __float_as_uint(s + 0.f);  // (-0 is 0)
  return (x >> 31) ? ~x : x | 0x80000000u;
}

// Exclusive prefix sums of two counts over the CTA.
__device__ __forceinline__ void block_prefix(int32_t& a, int32_t& b, int32_t (*sums)[2]) {
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
  for (int w = 0; w < warp; ++w) {
    before_a += sums[w][0];
    before_b += sums[w][1];
  }
  a = before_a + ia - a;
  b = before_b + ib - b;
}

// Keys of a thread's run of pages, i0 .. i1 - 1: in registers where the run is short.
struct Held {
  const uint32_t* keys;
  int32_t i0, i1;
  bool held;
  uint32_t k[kHeld];
  template <typename F>
  __device__ __forceinline__ void each(F&& f) const {
    if (held) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i0 + i < i1) f(i0 + i, k[i]);
    } else {
      for (int32_t i = i0; i < i1; ++i) f(i, keys[i]);
    }
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kRow = 2 * D + 32;  // bf16 elements between rows of q (64 bytes of padding: two rows of a load in different banks)
  constexpr int kChunks = 2 * D / 32, kPer = kBins / kThreads;
  extern __shared__ uint32_t keys[];  // of all pages, in the cluster's first CTA
  __shared__ __align__(16) __nv_bfloat16 qc[16 * kRow];
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t least[kWarps], most[kWarps], warp_sum[kWarps];
  __shared__ uint32_t pick[3];
  __shared__ int32_t sums[kWarps][2];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int32_t cta = static_cast<int32_t>(cluster_rank()), row = static_cast<int32_t>(blockIdx.x) / p.cluster;
  const int32_t t = row % p.T, bh = row / p.T, b = bh / p.Hkv, h = bh % p.Hkv;
  int32_t j0 = cta * kPassPages + warp * 8;  // this warp's pages; the quad's is j0 + g
  const int32_t step = p.cluster * kPassPages;
  // (the table's entries and q are on their way before the length is known)
  const int32_t* table = p.table + b * p.M;
  int32_t page = j0 + g < p.M ? table[j0 + g] : -1;
  const __nv_bfloat16* q = p.q + b * p.qs[0] + static_cast<int64_t>(h) * p.G * p.qs[1] + t * p.qs[2];
  uint32_t top = 0;
  for (int i = threadIdx.x; i < p.G * (D / 8); i += kThreads) {
    const uint4 x = *reinterpret_cast<const uint4*>(q + (i / (D / 8)) * p.qs[1] + i % (D / 8) * 8);
    const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    top = max(top, max(m & 0xFFFFu, m >> 16));
  }
  const int32_t n = pages_seen(p, b, t, cta == 0 && threadIdx.x == 0 && h == 0 ? p.err : nullptr);
  int32_t* index = p.index + static_cast<int64_t>(row) * p.keep;
  if (cta == 0)
    for (int32_t i = min(n, p.keep) + threadIdx.x; i < p.keep; i += kThreads) index[i] = -1;
  if (n <= p.keep) {  // (uniform over the cluster) all are kept: nothing to score
    if (cta == 0)
      for (int32_t i = threadIdx.x; i < n; i += kThreads) index[i] = i;
    return;
  }
  if (p.cluster > 1) cluster_arrive();  // (a CTA's shared memory is written once it is known to run)
  // ---- bounds: a pass of pages is on its way while the one before is scored
  uint4 x[kChunks];
  bool known;
  auto load = [&](int32_t j, uint4 (&y)[kChunks]) {  // the quad's page j, whose number is `page`; then the next number
    const bool in = j < n && page >= 0 && page < p.pages;
    if (j < n && !in && t4 == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
    const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(in ? page : 0) * p.Hkv + h) * 2 * D) + t4;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) y[c] = in ? src[c * 4] : make_uint4(0, 0, 0, 0);
    page = j + step < n ? table[j + step] : -1;
    return in;
  };
  known = load(j0 + g, x);
  // ---- the group's unit
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) warp_sum[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = max(top, warp_sum[w]);
  const float largest = __uint_as_float(top << 16);
  float unit = 0.f, inv = 0.f;  // (codes are 0 then)
  const bool usual = largest < kUsualTop;
  if (usual) unit_of(largest, 6, unit, inv);
  // codes of 16 q heads (a head once more in rows past the last one)
  auto code = [&](int32_t r0) {
    for (int i = threadIdx.x; i < 16 * (D / 8); i += kThreads) {
      const int r = i / (D / 8), d = i % (D / 8) * 8;
      const uint4 y = *reinterpret_cast<const uint4*>(q + min(r0 + r, p.G - 1) * p.qs[1] + d);
      const uint32_t w[4] = {y.x, y.y, y.z, y.w};
      uint32_t up[4], down[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = usual ? rintf(__uint_as_float(w[k] << 16) * inv) : 0.f, c = usual ? rintf(__uint_as_float(w[k] & 0xFFFF0000u) * inv) : 0.f;
        up[k] = pack_bf16x2(fmaxf(a, 0.f), fmaxf(c, 0.f));
        down[k] = pack_bf16x2(fminf(a, 0.f), fminf(c, 0.f));
      }
      *reinterpret_cast<uint4*>(&qc[r * kRow + d]) = make_uint4(up[0], up[1], up[2], up[3]);
      *reinterpret_cast<uint4*>(&qc[r * kRow + D + d]) = make_uint4(down[0], down[1], down[2], down[3]);
    }
    __syncthreads();
  };
  uint32_t first_keys;  // the first CTA's `keys`
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(first_keys) : "r"(smem_u32(keys)), "r"(0));
  bool started = p.cluster == 1;
  for (int32_t pass = 0; pass * step < n; ++pass) {  // (as many for every CTA of the cluster)
    uint4 ahead[kChunks];
    const bool known_ahead = load(j0 + step + g, ahead);
    float best[2] = {-INFINITY, -INFINITY};  // pages 2 t4 and 2 t4 + 1 of the warp's
    for (int32_t r0 = 0; r0 < p.G; r0 += 16) {
      if (pass == 0 || p.G > 16) {
        if (pass + r0 > 0) __syncthreads();
        code(r0);
      }
      float acc[2][4] = {};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint4 lo = *reinterpret_cast<const uint4*>(&qc[g * kRow + c * 32 + t4 * 8]);
        const uint4 hi = *reinterpret_cast<const uint4*>(&qc[(g + 8) * kRow + c * 32 + t4 * 8]);
        mma_bf16(acc[0], lo.x, hi.x, lo.y, hi.y, x[c].x, x[c].y);
        mma_bf16(acc[1], lo.z, hi.z, lo.w, hi.w, x[c].z, x[c].w);
      }
      // heads g and g + 8
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float s0 = acc[0][k] + acc[1][k], s1 = acc[0][k + 2] + acc[1][k + 2];
        best[k] = fmaxf(best[k], fmaxf(fabsf(s0) < INFINITY ? s0 : INFINITY, fabsf(s1) < INFINITY ? s1 : INFINITY));
      }
    }
    if (!started) cluster_wait();
    started = true;
    const uint32_t ok = __ballot_sync(0xffffffffu, known);  // lane 4 g stands for page g
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) best[k] = fmaxf(best[k], __shfl_xor_sync(0xffffffffu, best[k], o));
      const int32_t i = 2 * t4 + k;
      if (g == 0 && j0 + i < n)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(first_keys + 4 * (j0 + i)), "r"(ordered(ok >> (4 * i) & 1u ? best[k] : -INFINITY)) : "memory");
    }
#pragma unroll
    for (int c = 0; c < kChunks; ++c) x[c] = ahead[c];
    known = known_ahead;
    j0 += step;
  }
  if (p.cluster > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (cta > 0) return;
  // ---- the choice (n is above keep, which is at least first + recent: pages m0 .. m1 - 1 are chosen by their keys)
  const int32_t m0 = p.first, m1 = n - p.recent;
  uint32_t want = static_cast<uint32_t>(p.keep - p.first - p.recent);
  for (int32_t i = threadIdx.x; i < p.first; i += kThreads) index[i] = i;
  for (int32_t i = threadIdx.x; i < p.recent; i += kThreads) index[p.keep - p.recent + i] = m1 + i;
  if (want == 0) return;
#pragma unroll
  for (int i = 0; i < kPer; ++i) hist[i * kThreads + threadIdx.x] = 0;
  __syncthreads();  // (a lone CTA's own keys)
  // a run of pages a thread (odd: a warp's runs start in different banks)
  const int32_t per = (m1 - m0 + kThreads - 1) / kThreads | 1;
  Held mine;
  mine.keys = keys;
  mine.i0 = m0 + static_cast<int32_t>(threadIdx.x) * per;
  mine.i1 = min(mine.i0 + per, m1);
  mine.held = per <= kHeld;
  if (mine.held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) mine.k[i] = mine.i0 + i < mine.i1 ? keys[mine.i0 + i] : 0u;
  }
  // the range of the keys: its digits, not the floats', spread them over the bins
  uint32_t lo = ~0u, hi = 0u;
  mine.each([&](int32_t, uint32_t k) {
    lo = min(lo, k);
    hi = max(hi, k);
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    least[warp] = lo;
    most[warp] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = min(lo, least[w]);
    hi = max(hi, most[w]);
  }
  // the least kept key, from its highest digit on: of key - lo, the bits above `shift` are `digits`, and of the pages that
  // share them `want` are kept
  int shift = 32 - __clz(hi - lo);
  uint32_t digits = 0;
  bool all = shift == 0;  // (equal keys)
  while (!all) {
    const int bits = min(shift, 11);
    shift -= bits;
    mine.each([&](int32_t, uint32_t k) {
      const uint32_t y = (k - lo) >> shift;
      if (y >> bits == digits) atomicAdd(&hist[y & ((1u << bits) - 1)], 1u);
    });
    __syncthreads();
    // suffix sums: thread i has kPer bins, counted from the top
    const int first_bin = kBins - 1 - kPer * static_cast<int>(threadIdx.x);
    uint32_t c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      sum += c[i] = hist[first_bin - i];
      hist[first_bin - i] = 0;
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t above = inc - sum;
    for (int w = 0; w < warp; ++w) above += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < want && want <= above + c[i]) {
        pick[0] = first_bin - i;
        pick[1] = want - above;
        pick[2] = c[i];
      }
      above += c[i];
    }
    __syncthreads();
    digits = digits << bits | pick[0];
    want = pick[1];
    all = shift == 0 || pick[2] == want;
  }
  // kept pages in order: those above the least digits, and the first `want` ones at them
  int32_t more = 0, same = 0;
  mine.each([&](int32_t, uint32_t k) {
    const uint32_t y = (k - lo) >> shift;
    more += y > digits;
    same += y == digits;
  });
  block_prefix(more, same, sums);
  index += p.first;
  mine.each([&](int32_t i, uint32_t k) {
    const uint32_t y = (k - lo) >> shift;
    if (y > digits) {
      index[more++ + min(same, static_cast<int32_t>(want))] = i;
    } else if (y == digits) {
      if (same < static_cast<int32_t>(want)) index[more + same] = i;
      ++same;
    }
  });
}

template <int D>
bsa_status launch(const SelectParams& p, cudaStream_t stream) {
  const bsa_status st = ensure_smem_attr(reinterpret_cast<const void*>(select_kernel<D>), kMaxPages * sizeof(uint32_t), "set page selection smem size");
  if (st != BSA_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.Hkv * p.T * p.cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.M) * sizeof(uint32_t);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, select_kernel<D>, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged select launch");
  return BSA_OK;
}

}  // namespace

bool paged_select_fits(const bsa_paged_select_args* a) {
  return a->M <= kMaxPages && static_cast<int64_t>(a->B) * a->cache.Hkv <= INT32_MAX / kMaxCluster / a->T;
}

bsa_status paged_select_launch(const bsa_paged_select_args* a, cudaStream_t stream) {
  SelectParams p{};
  p.bounds = static_cast<const __nv_bfloat16*>(a->cache.bounds);
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  for (int i = 0; i < 3; ++i) p.qs[i] = a->q_stride[i];
  p.table = a->table;
  p.lens = a->lens;
  p.q_lens = a->q_lens;
  p.index = a->index;
  p.B = a->B;
  p.Hkv = a->cache.Hkv;
  p.G = a->Hq / a->cache.Hkv;
  p.T = static_cast<int32_t>(a->T);
  p.shift = page_shift(a->cache.page);
  p.pages = static_cast<int32_t>(a->cache.pages);
  p.M = a->M;
  p.keep = static_cast<int32_t>(a->keep);
  p.first = static_cast<int32_t>(a->first);
  p.recent = static_cast<int32_t>(a->recent);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  // CTAs a query: more while all of them have an SM to themselves and a pass of pages each (selection and attention by 1, 2,
  // 4 and 8: 8 queries of 2048 pages 48, 39, 34 and 31 us, 32 of 512 33.9, 31.9, 30.5 and 37, 128 of up to 512 56, 62, 70 and 86)
  const int64_t queries = static_cast<int64_t>(p.B) * p.Hkv * p.T;
  p.cluster = 1;
  while (p.cluster < kMaxCluster && queries * p.cluster * 2 <= num_sms() && p.cluster * kPassPages < p.M) p.cluster *= 2;
  return a->cache.D == 128 ? launch<128>(p, stream) : launch<64>(p, stream);
}

}  // namespace bsa
