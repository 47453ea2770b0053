// The pages worth attending to, for each query: those with the largest bound on q.k.
//
// A page's keys lie between its bounds, so sum_d max(q_d hi_d, q_d lo_d) bounds q.k over the page.  With q+ =
// max(q, 0) and q- = min(q, 0) that is q+ hi + q- lo: one matrix product of length 2 D, [q+ | q-] [hi | lo]^T.
//
// Exactness.  q is taken as whole numbers of up to 8 bits (|qc| <= 128, times 2^f), the bounds are whole numbers
// |c| <= 256 times 2^e of the page.  Products are at most 2^15, their sums over D <= 128 channels (of a channel's two products
// one is 0) at most 2^22: multiples of 2^e that fp32 accumulators hold exactly, whatever the order.  2^f is the same for all of a
// query's pages and is left out.  So the choice is one and the same for every way to split the work, and ties are real ties.
//
// First kernel: a warp scores 8 pages at a time as the narrow side of m16n8k16 products, the group's q heads being
// the 16-row side.  The channels of a product's k axis are taken in an order that makes a thread's share of 8 pages 16-byte loads
// straight from memory (thread t of a quad: channels 8 t .. 8 t + 7 of every 32), the four of a quad 64 bytes
// side by side; nothing goes through shared memory but q.
// Second kernel: one CTA a query.  Scores as ordered 32-bit keys, less the smallest; counts of their digits, from the
// highest one on, give the least key that is kept and how many pages of it; then the kept pages in order, by
// prefix sums.
#include <algorithm>

#include "paged.cuh"

namespace bsa {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScorePages = kScoreThreads / 4;  // pages of one CTA: 8 a warp
constexpr int kPickThreads = 512;
constexpr int kBins = 2048;
constexpr int kHeld = 8;  // keys a thread keeps in registers

struct SelectParams {
  const __nv_bfloat16* bounds;
  const __nv_bfloat16* q;
  int64_t qs[3];
  const int32_t *table, *lens, *q_lens;
  int32_t* index;
  uint32_t* keys;  // [B, Hkv, T, M]
  int32_t B, Hkv, G, T, shift, pages;
  int64_t M;
  int32_t keep, first, recent;
  int32_t chunks;  // CTAs that score a query's pages
  uint32_t* err;
};

// Pages that token t of sequence b sees (0: padding).
__device__ __forceinline__ int32_t pages_seen(const SelectParams& p, int32_t b, int32_t t, uint32_t* err) {
  const int32_t len = paged_len(p.lens[b], p.M << p.shift, err);
  const int32_t nq = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
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

template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kRow = 2 * D + 32;  // bf16 elements between rows of q (64 bytes of padding: two rows of a load in different banks)
  constexpr int kChunks = 2 * D / 32;
  __shared__ __align__(16) __nv_bfloat16 qc[16 * kRow];
  __shared__ uint32_t tops[kScoreThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int32_t row = static_cast<int32_t>(blockIdx.x) / p.chunks, chunk = static_cast<int32_t>(blockIdx.x) % p.chunks;
  const int32_t t = row % p.T, bh = row / p.T, b = bh / p.Hkv, h = bh % p.Hkv;
  const int32_t j0 = chunk * kScorePages + warp * 8, j = j0 + g;  // this warp's pages, this quad's
  // (the table's entry and q are on their way before the length is known)
  const int32_t page = j < p.M ? p.table[b * p.M + j] : -1;
  const __nv_bfloat16* q = p.q + b * p.qs[0] + static_cast<int64_t>(h) * p.G * p.qs[1] + t * p.qs[2];
  uint32_t top = 0;
  for (int i = threadIdx.x; i < p.G * (D / 8); i += kScoreThreads) {
    const uint4 x = *reinterpret_cast<const uint4*>(q + (i / (D / 8)) * p.qs[1] + i % (D / 8) * 8);
    const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    top = max(top, max(m & 0xFFFFu, m >> 16));
  }
  const int32_t n = pages_seen(p, b, t, chunk == 0 && threadIdx.x == 0 && h == 0 ? p.err : nullptr);
  if (chunk * kScorePages >= n || n <= p.keep) return;  // (all are kept: nothing to score)
  const bool known = j < n && page >= 0 && page < p.pages;
  if (j < n && !known && t4 == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
  const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(known ? page : 0) * p.Hkv + h) * 2 * D) + t4;
  uint4 x[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) x[c] = known ? src[c * 4] : make_uint4(0, 0, 0, 0);
  // ---- the group's unit
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScoreThreads / 32; ++w) top = max(top, tops[w]);
  const float largest = __uint_as_float(top << 16);
  float unit = 0.f, inv = 0.f;  // (codes are 0 then)
  const bool usual = largest < kUsualTop;
  if (usual) unit_of(largest, 6, unit, inv);
  float best[2] = {-INFINITY, -INFINITY};  // pages 2 t4 and 2 t4 + 1 of the warp's
  for (int32_t r0 = 0; r0 < p.G; r0 += 16) {
    // ---- codes of 16 q heads (a head once more in rows past the last one)
    if (r0 > 0) __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 8); i += kScoreThreads) {
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
  const uint32_t ok = __ballot_sync(0xffffffffu, known);  // lane 4 g stands for page g
  uint32_t* keys = p.keys + static_cast<int64_t>(row) * p.M;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int o = 4; o < 32; o *= 2) best[k] = fmaxf(best[k], __shfl_xor_sync(0xffffffffu, best[k], o));
    const int32_t i = 2 * t4 + k;
    if (g == 0 && j0 + i < n) keys[j0 + i] = ordered(ok >> (4 * i) & 1u ? best[k] : -INFINITY);
  }
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

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kWarps = kPickThreads / 32, kPer = kBins / kPickThreads;
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t least[kWarps], most[kWarps], warp_sum[kWarps];
  __shared__ uint32_t pick[3];
  __shared__ int32_t sums[kWarps][2];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = blockIdx.x;
  const int32_t t = static_cast<int32_t>(row % p.T), b = static_cast<int32_t>(row / p.T / p.Hkv);
  const int32_t n = pages_seen(p, b, t, nullptr), kept = min(n, p.keep);
  int32_t* index = p.index + row * p.keep;
  for (int32_t i = kept + threadIdx.x; i < p.keep; i += kPickThreads) index[i] = -1;
  if (n <= p.keep) {
    for (int32_t i = threadIdx.x; i < n; i += kPickThreads) index[i] = i;
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (n is above keep, which is at least first + recent: pages m0 .. m1 - 1 are chosen by their keys)
  const int32_t m0 = p.first, m1 = n - p.recent;
  uint32_t want = static_cast<uint32_t>(p.keep - p.first - p.recent);
  Held mine;
  const int32_t per = (m1 - m0 + kPickThreads - 1) / kPickThreads;
  mine.keys = p.keys + row * p.M;
  mine.i0 = m0 + static_cast<int32_t>(threadIdx.x) * per;
  mine.i1 = min(mine.i0 + per, m1);
  mine.held = per <= kHeld;
  if (mine.held) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) mine.k[i] = mine.i0 + i < mine.i1 ? mine.keys[mine.i0 + i] : 0u;
  }
  for (int32_t i = threadIdx.x; i < p.first; i += kPickThreads) index[i] = i;
  for (int32_t i = threadIdx.x; i < p.recent; i += kPickThreads) index[p.keep - p.recent + i] = m1 + i;
  if (want == 0) return;
  // ---- the range of the keys: its digits, not the floats', spread them over the bins
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
#pragma unroll
  for (int i = 0; i < kPer; ++i) hist[i * kPickThreads + threadIdx.x] = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    lo = min(lo, least[w]);
    hi = max(hi, most[w]);
  }
  // ---- the least kept key, from its highest digit on: of key - lo, the bits above `shift` are `digits`, and of the pages
  // that share them `want` are kept
  int shift = 32 - __clz(hi - lo);
  uint32_t digits = 0;
  bool all = shift == 0;  // (equal keys)
  while (!all) {
    const int bits = min(shift, 11);
    shift -= bits;
    mine.each([&](int32_t, uint32_t k) {
      const uint32_t x = (k - lo) >> shift;
      if (x >> bits == digits) atomicAdd(&hist[x & ((1u << bits) - 1)], 1u);
    });
    __syncthreads();
    // suffix sums: thread i has kPer bins, counted from the top
    const int top = kBins - 1 - kPer * static_cast<int>(threadIdx.x);
    uint32_t c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      sum += c[i] = hist[top - i];
      hist[top - i] = 0;
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t above = inc - sum;
    for (int w = 0; w < warp; ++w) above += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < want && want <= above + c[i]) {
        pick[0] = top - i;
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
  // ---- kept pages in order: those above the least digits, and the first `want` ones at them
  int32_t more = 0, same = 0;
  mine.each([&](int32_t, uint32_t k) {
    const uint32_t x = (k - lo) >> shift;
    more += x > digits;
    same += x == digits;
  });
  block_prefix(more, same, sums);
  index += p.first;
  mine.each([&](int32_t i, uint32_t k) {
    const uint32_t x = (k - lo) >> shift;
    if (x > digits) {
      index[more++ + min(same, static_cast<int32_t>(want))] = i;
    } else if (x == digits) {
      if (same < static_cast<int32_t>(want)) index[more + same] = i;
      ++same;
    }
  });
}

}  // namespace

static int64_t score_chunks(const bsa_paged_select_args* a) { return (a->M + kScorePages - 1) / kScorePages; }

bool paged_select_fits(const bsa_paged_select_args* a) {
  return score_chunks(a) <= INT32_MAX / (static_cast<int64_t>(a->B) * a->cache.Hkv * a->T);
}

size_t paged_select_workspace_bytes(const bsa_paged_select_args* a) {
  return static_cast<size_t>(a->B) * a->cache.Hkv * a->T * a->M * sizeof(uint32_t);
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
  p.keys = static_cast<uint32_t*>(a->workspace);
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
  cudaError_t e;
  p.chunks = static_cast<int32_t>(score_chunks(a));
  const dim3 grid(static_cast<unsigned>(p.chunks * a->B * a->cache.Hkv * a->T));
  e = a->cache.D == 128 ? launch_kernel(score_kernel<128>, grid, dim3(kScoreThreads), 0, stream, p)
                        : launch_kernel(score_kernel<64>, grid, dim3(kScoreThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged score launch");
  e = launch_kernel(pick_kernel, dim3(static_cast<unsigned>(a->B * a->cache.Hkv * a->T)), dim3(kPickThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged select launch");
  return BSA_OK;
}

}  // namespace bsa
