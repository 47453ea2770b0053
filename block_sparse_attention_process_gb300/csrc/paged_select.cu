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
// Second kernel: one CTA a query.  Scores as ordered 32-bit keys; three digits' counts give the least key that is
// kept and how many pages of it; then the kept pages in order, by prefix sums.
#include <algorithm>

#include "paged.cuh"

namespace bsa {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kScorePages = 128;  // pages of one CTA
constexpr int kPickThreads = 512;
constexpr int kBins = 2048;

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

// Order of scores as order of unsigned numbers; above every score: all ones.
__device__ __forceinline__ uint32_t ordered(float s) {
  const uint32_t x = __float_as_uint(s + 0.f);  // (-0 is 0)
  return (x >> 31) ? ~x : x | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const __grid_constant__ SelectParams p) {
  constexpr int kRow = 2 * D + 32;  // bf16 elements between rows of q (64 bytes of padding: two rows of a load in different banks)
  constexpr int kChunks = 2 * D / 32;
  __shared__ __align__(16) __nv_bfloat16 qc[16 * kRow];
  __shared__ float score[kScorePages];
  __shared__ uint32_t tops[kScoreThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
  const int32_t row = static_cast<int32_t>(blockIdx.x) / p.chunks, chunk = static_cast<int32_t>(blockIdx.x) % p.chunks;
  const int32_t t = row % p.T, bh = row / p.T, b = bh / p.Hkv, h = bh % p.Hkv;
  const int32_t n = pages_seen(p, b, t, chunk == 0 && threadIdx.x == 0 && h == 0 ? p.err : nullptr);
  const int32_t j0 = chunk * kScorePages;
  if (j0 >= n || n <= p.keep) return;  // (all are kept: nothing to score)
  const __nv_bfloat16* q = p.q + b * p.qs[0] + static_cast<int64_t>(h) * p.G * p.qs[1] + t * p.qs[2];
  // ---- the group's unit
  uint32_t top = 0;
  for (int i = threadIdx.x; i < p.G * (D / 8); i += kScoreThreads) {
    const uint4 x = *reinterpret_cast<const uint4*>(q + (i / (D / 8)) * p.qs[1] + i % (D / 8) * 8);
    const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
    top = max(top, max(m & 0xFFFFu, m >> 16));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (lane == 0) tops[warp] = top;
  for (int i = threadIdx.x; i < kScorePages; i += kScoreThreads) score[i] = -INFINITY;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScoreThreads / 32; ++w) top = max(top, tops[w]);
  const float largest = __uint_as_float(top << 16);
  float unit = 0.f, inv = 0.f;  // (codes are 0 then)
  const bool usual = largest < kUsualTop;
  if (usual) unit_of(largest, 6, unit, inv);
  for (int32_t r0 = 0; r0 < p.G; r0 += 16) {
    // ---- codes of 16 q heads (a head once more in rows past the last one)
    if (r0 > 0) __syncthreads();
    for (int i = threadIdx.x; i < 16 * (D / 8); i += kScoreThreads) {
      const int r = i / (D / 8), d = i % (D / 8) * 8;
      const uint4 x = *reinterpret_cast<const uint4*>(q + min(r0 + r, p.G - 1) * p.qs[1] + d);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
    for (int32_t i = warp * 8; i < kScorePages && j0 + i < n; i += kScoreThreads / 32 * 8) {
      const int32_t j = j0 + i + g;
      const int32_t page = j < n ? p.table[b * p.M + j] : -1;
      const bool known = page >= 0 && page < p.pages;
      if (j < n && !known && t4 == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
      const uint4* src = reinterpret_cast<const uint4*>(p.bounds + (static_cast<int64_t>(known ? page : 0) * p.Hkv + h) * 2 * D) + t4;
      uint4 x[kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; ++c) x[c] = known ? __ldg(src + c * 4) : make_uint4(0, 0, 0, 0);
      float acc[2][4] = {};
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint4 lo = *reinterpret_cast<const uint4*>(&qc[g * kRow + c * 32 + t4 * 8]);
        const uint4 hi = *reinterpret_cast<const uint4*>(&qc[(g + 8) * kRow + c * 32 + t4 * 8]);
        mma_bf16(acc[0], lo.x, hi.x, lo.y, hi.y, x[c].x, x[c].y);
        mma_bf16(acc[1], lo.z, hi.z, lo.w, hi.w, x[c].z, x[c].w);
      }
      // pages 2 t4 and 2 t4 + 1, heads g and g + 8
      float best[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float s0 = acc[0][k] + acc[1][k], s1 = acc[0][k + 2] + acc[1][k + 2];
        best[k] = fmaxf(fabsf(s0) < INFINITY ? s0 : INFINITY, fabsf(s1) < INFINITY ? s1 : INFINITY);
#pragma unroll
        for (int o = 4; o < 32; o *= 2) best[k] = fmaxf(best[k], __shfl_xor_sync(0xffffffffu, best[k], o));
      }
      const uint32_t ok = __ballot_sync(0xffffffffu, known);  // lane 4 g stands for page g
      if (g == 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (ok >> (4 * (2 * t4 + k)) & 1u) score[i + 2 * t4 + k] = fmaxf(score[i + 2 * t4 + k], best[k]);
      }
    }
  }
  __syncthreads();
  uint32_t* keys = p.keys + static_cast<int64_t>(row) * p.M;
  for (int32_t i = threadIdx.x; i < kScorePages && j0 + i < n; i += kScoreThreads) {
    const int32_t j = j0 + i;
    keys[j] = j < p.first || j >= n - p.recent ? ~0u : ordered(score[i]);
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

__global__ void __launch_bounds__(kPickThreads) pick_kernel(const __grid_constant__ SelectParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sum[kPickThreads / 32];
  __shared__ uint32_t pick[2];
  __shared__ int32_t sums[kPickThreads / 32][2];
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
  const uint32_t* keys = p.keys + row * p.M;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // ---- the least kept key, from its highest digit on
  uint32_t prefix = 0, mask = 0;
  uint32_t want = kept;  // of the keys that share the prefix, this many largest ones are kept
  constexpr int kShift[3] = {21, 10, 0};
#pragma unroll
  for (int digit = 0; digit < 3; ++digit) {
    const int bits = digit == 2 ? 10 : 11, shift = kShift[digit];
    for (int i = threadIdx.x; i < kBins; i += kPickThreads) hist[i] = 0;
    __syncthreads();
    for (int32_t i = threadIdx.x; i < n; i += kPickThreads) {
      const uint32_t k = keys[i];
      if ((k & mask) == prefix) atomicAdd(&hist[k >> shift & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    // suffix sums: thread i has bins 4 i .. 4 i + 3, counted from the top
    constexpr int kPer = kBins / kPickThreads;
    const int top = kBins - 1 - kPer * static_cast<int>(threadIdx.x);
    uint32_t c[kPer], mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += c[i] = hist[top - i];
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    uint32_t above = inc - mine;
    for (int w = 0; w < warp; ++w) above += warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (above < want && want <= above + c[i]) {
        pick[0] = top - i;
        pick[1] = want - above;
      }
      above += c[i];
    }
    __syncthreads();
    prefix |= pick[0] << shift;
    mask |= ((1u << bits) - 1) << shift;
    want = pick[1];
    __syncthreads();
  }
  // ---- kept pages in order: those above the least key, and the first `want` ones at it; a run of pages a thread
  const int32_t per = (n + kPickThreads - 1) / kPickThreads, i0 = static_cast<int32_t>(threadIdx.x) * per, i1 = min(i0 + per, n);
  int32_t more = 0, same = 0;
  for (int32_t i = i0; i < i1; ++i) {
    const uint32_t k = keys[i];
    more += k > prefix;
    same += k == prefix;
  }
  block_prefix(more, same, sums);
  for (int32_t i = i0; i < i1; ++i) {
    const uint32_t k = keys[i];
    if (k > prefix) {
      index[more++ + min(same, static_cast<int32_t>(want))] = i;
    } else if (k == prefix) {
      if (same < static_cast<int32_t>(want)) index[more + same] = i;
      ++same;
    }
  }
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
