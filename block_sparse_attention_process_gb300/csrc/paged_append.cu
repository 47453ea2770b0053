// Keys and values into the slots of the cache in pages, and the bounds of the pages' keys.
//
// Without bounds a row (one token and head) is D/8 lanes of 16 bytes, wherever its slot is.
//
// With bounds a warp, or two or four, takes the tokens of one sequence and head that go into one page: the slots of a sequence's
// tokens follow each other, so token t lies at place (o + t) % page, o being the place of token 0, and
// unit u holds tokens u * page - o .. (u + 1) * page - o - 1.  It writes them, reads the keys that the page held before them, and
// has every key of the page in registers then: maxima and minima are exact in any order, so the bounds need no
// atomics, no second pass over the new keys, and come out the same each time.  Where a place among the new tokens' was left out
// (padding, or a slot elsewhere) the page holds a key there that no register does: its bounds are infinite then.
// 4 x 8 heads x 8191 tokens: 44.0 us with bounds (pages of 64; 44.8 with pages of 16, 48.1 of 256), 42.8 without: 90 to 92% of a
// copy's bandwidth.  64 x 8 heads x 1 token: 3.6 and 2.1 us, latency.
#include <algorithm>

#include "paged.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 128;  // (256: 54 us for 4 x 8 x 8191 tokens, 128: 44)
constexpr int kWarpPlaces = 16;
constexpr int kBatch = 4;      // rows that a thread has on their way at a time

struct AppendParams {
  bsa_paged_cache c;
  const __nv_bfloat16 *k, *v;
  int64_t ks[3], vs[3];
  const int32_t* slots;
  int32_t B, shift;
  int64_t T;
  int64_t units;  // of one sequence and head
  uint32_t* err;
};

__device__ __forceinline__ int64_t page_at(const int64_t (&stride)[3], int32_t slot, int32_t shift, int32_t h) {
  return (slot >> shift) * stride[0] + h * stride[1] + (slot & ((1 << shift) - 1)) * stride[2];
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_rows_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8;
  griddep_launch_dependents();
  griddep_wait();
  constexpr uint32_t kSubs = kThreads / kLanes;
  const int u = threadIdx.x % kLanes;
  const uint32_t T = static_cast<uint32_t>(p.T), rows = static_cast<uint32_t>(p.B) * p.c.Hkv * T;  // (below 2^31)
  const int64_t limit = p.c.pages << p.shift;
  // rows in order of (b, h, t), kBatch at a time
  for (uint32_t r0 = blockIdx.x * kBatch * kSubs + threadIdx.x / kLanes; r0 < rows; r0 += gridDim.x * kBatch * kSubs) {
    int32_t slot[kBatch], h[kBatch];
    uint4 k[kBatch], v[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const uint32_t r = r0 + x * kSubs;
      slot[x] = -1;
      if (r >= rows) continue;
      const uint32_t bh = r / T, t = r - bh * T, b = bh / p.c.Hkv;
      h[x] = static_cast<int32_t>(bh - b * p.c.Hkv);
      slot[x] = p.slots[b * T + t];
      // (read before the slot is known: it is the call's own memory)
      k[x] = __ldcs(reinterpret_cast<const uint4*>(p.k + b * p.ks[0] + h[x] * p.ks[1] + t * p.ks[2] + 8 * u));
      v[x] = __ldcs(reinterpret_cast<const uint4*>(p.v + b * p.vs[0] + h[x] * p.vs[1] + t * p.vs[2] + 8 * u));
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      if (slot[x] < 0) continue;
      if (slot[x] >= limit) {
        if (u == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
        continue;
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.c.k) + page_at(p.c.k_stride, slot[x], p.shift, h[x]) + 8 * u) = k[x];
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.c.v) + page_at(p.c.v_stride, slot[x], p.shift, h[x]) + 8 * u) = v[x];
    }
  }
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Running maximum and minimum of 8 channels, and the largest magnitude as bf16 bits (NaN is above every number there).
struct Range {
  float hi[8], lo[8];
  uint32_t top;
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = -INFINITY;
      lo[i] = INFINITY;
    }
    top = 0;
  }
  __device__ __forceinline__ void add(const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[2 * i] = fmaxf(hi[2 * i], lo_f(w[i]));
      hi[2 * i + 1] = fmaxf(hi[2 * i + 1], hi_f(w[i]));
      lo[2 * i] = fminf(lo[2 * i], lo_f(w[i]));
      lo[2 * i + 1] = fminf(lo[2 * i + 1], hi_f(w[i]));
      m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    }
    top = max(top, max(m & 0xFFFFu, m >> 16));
  }
};

// The warps that share a page (1, 2 or 4).
__device__ __forceinline__ void group_sync(int group, int warps) {
  if (warps == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}
__device__ __forceinline__ bool group_any(int group, int warps, bool x) {
  if (warps == 1) return __any_sync(0xffffffffu, x);
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(x)), "r"(group + 1), "r"(warps * 32)
      : "memory");
  return any != 0u;
}

template <int D, int warps>
__global__ void __launch_bounds__(kThreads) append_bounds_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 8, kWarps = kThreads / 32;
  __shared__ float hi[kWarps][D], lo[kWarps][D];
  __shared__ uint32_t top[kWarps];
  __shared__ int32_t left_out[kWarps], stored[kWarps];  // the first place left out, the last one stored
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kSubs = warps * (32 / kLanes);
  const int group = warp / warps, first_warp = group * warps;
  const int u = lane % kLanes, sub = (warp - first_warp) * (32 / kLanes) + lane / kLanes;
  const int32_t page = 1 << p.shift;
  const int64_t limit = p.c.pages << p.shift;
  const uint32_t at = blockIdx.x * (kWarps / warps) + group;  // (below 2^31)
  if (at >= static_cast<uint32_t>(p.units) * p.B * p.c.Hkv) return;
  const uint32_t bh = at / static_cast<uint32_t>(p.units), unit = at - bh * static_cast<uint32_t>(p.units);
  const int32_t b = static_cast<int32_t>(bh / p.c.Hkv), h = static_cast<int32_t>(bh) - b * p.c.Hkv;
  const int32_t* slots = p.slots + b * p.T;
  const int32_t s0 = slots[0];
  const int32_t o = s0 < 0 ? 0 : s0 & (page - 1);
  const int64_t t0 = static_cast<int64_t>(unit) * page - o;  // token of the page's place 0
  if (t0 >= p.T) return;
  // the page is that of the unit's first token
  const int32_t first = slots[max(t0, static_cast<int64_t>(0))];
  const int32_t begin = t0 < 0 ? o : 0;  // its place
  const int32_t page0 = first < 0 || first >= limit ? -1 : first - begin;  // slot of place 0 (another place: nothing fits)
  const bool good = page0 >= 0 && (page0 & (page - 1)) == 0;
  Range r;
  r.clear();
  int32_t last = -1, gap = INT32_MAX;
  bool wrong = false;
  const __nv_bfloat16* src_k = p.k + b * p.ks[0] + h * p.ks[1] + 8 * u;
  const __nv_bfloat16* src_v = p.v + b * p.vs[0] + h * p.vs[1] + 8 * u;
  __nv_bfloat16* dst_k = static_cast<__nv_bfloat16*>(p.c.k) + 8 * u;
  __nv_bfloat16* dst_v = static_cast<__nv_bfloat16*>(p.c.v) + 8 * u;
  for (int32_t i0 = begin + sub; i0 < page && t0 + i0 < p.T; i0 += kBatch * kSubs) {
    int32_t slot[kBatch];
    uint4 k[kBatch], v[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int32_t i = i0 + x * kSubs;
      const bool in = i < page && t0 + i < p.T;
      slot[x] = in ? slots[t0 + i] : -1;
      // (read before the slot is known: it is the call's own memory)
      if (in) {
        k[x] = __ldcs(reinterpret_cast<const uint4*>(src_k + (t0 + i) * p.ks[2]));
        v[x] = __ldcs(reinterpret_cast<const uint4*>(src_v + (t0 + i) * p.vs[2]));
      }
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int32_t i = i0 + x * kSubs;
      if (slot[x] < 0 || !good || slot[x] != page0 + i) {
        wrong |= slot[x] >= 0;
        gap = min(gap, i);
        continue;
      }
      slot[x] = BSA_RANGE(slot[x], 0, static_cast<int32_t>(limit), p.err);
      *reinterpret_cast<uint4*>(dst_k + page_at(p.c.k_stride, slot[x], p.shift, h)) = k[x];
      *reinterpret_cast<uint4*>(dst_v + page_at(p.c.v_stride, slot[x], p.shift, h)) = v[x];
      r.add(k[x]);
      last = i;
    }
  }
  if (wrong && u == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
  if (!group_any(group, warps, last >= 0)) return;  // nothing stored
  // keys that the page held (places before the first new one)
  for (int32_t i = sub; i < begin; i += kSubs) r.add(*reinterpret_cast<const uint4*>(dst_k + page_at(p.c.k_stride, page0 + i, p.shift, h)));
  // ---- over the warp's rows, then over the warps
#pragma unroll
  for (int s = kLanes; s < 32; s *= 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.hi[i] = fmaxf(r.hi[i], __shfl_xor_sync(0xffffffffu, r.hi[i], s));
      r.lo[i] = fminf(r.lo[i], __shfl_xor_sync(0xffffffffu, r.lo[i], s));
    }
  }
  r.top = __reduce_max_sync(0xffffffffu, r.top);
  last = __reduce_max_sync(0xffffffffu, last);
  gap = __reduce_min_sync(0xffffffffu, gap);
  if (lane < kLanes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[warp][8 * u + i] = r.hi[i];
      lo[warp][8 * u + i] = r.lo[i];
    }
  }
  if (lane == 0) {
    top[warp] = r.top;
    left_out[warp] = gap;
    stored[warp] = last;
  }
  group_sync(group, warps);
  for (int d = threadIdx.x - first_warp * 32; d < D; d += warps * 32) {
    float a = hi[first_warp][d], c = lo[first_warp][d];
    uint32_t m = top[first_warp];
    gap = left_out[first_warp];
    last = stored[first_warp];
    for (int w = first_warp + 1; w < first_warp + warps; ++w) {
      a = fmaxf(a, hi[w][d]);
      c = fminf(c, lo[w][d]);
      m = max(m, top[w]);
      gap = min(gap, left_out[w]);
      last = max(last, stored[w]);
    }
    const bool whole = last < gap;
    if (!whole && d == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
    const float largest = __uint_as_float(m << 16);
    if (largest < kUsualTop && whole) {
      float s, inv;
      unit_of(largest, 7, s, inv);
      const float up = ceilf(a * inv) * s, down = floorf(c * inv) * s;
      a = up < a ? s : up;  // (a product that underflowed to 0)
      c = down > c ? -s : down;
    } else {
      a = INFINITY;
      c = -INFINITY;
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.c.bounds) + ((static_cast<int64_t>(page0 >> p.shift) * p.c.Hkv + h) * 2) * D + d;
    out[0] = __float2bfloat16_rn(a);
    out[D] = __float2bfloat16_rn(c);
  }
}

}  // namespace

int64_t paged_append_units(const bsa_paged_append_args* a) {
  return (a->T + 2 * a->cache.page - 2) / a->cache.page;  // (pages that T tokens in a row can lie in)
}

bsa_status paged_append_launch(const bsa_paged_append_args* a, cudaStream_t stream) {
  AppendParams p{};
  p.c = a->cache;
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = a->src_k_stride[i];
    p.vs[i] = a->src_v_stride[i];
  }
  p.slots = a->slots;
  p.B = a->B;
  p.shift = page_shift(a->cache.page);
  p.T = a->T;
  p.units = paged_append_units(a);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  cudaError_t e;
  if (a->cache.bounds) {
    // a warp for every kWarpPlaces places of a page, up to a CTA
    const int warps = std::min(a->cache.page / kWarpPlaces, kThreads / 32);
    const int64_t units = p.units * a->B * a->cache.Hkv, per = kThreads / 32 / warps;
    const dim3 grid(static_cast<unsigned>((units + per - 1) / per));
    auto kern = a->cache.D == 128 ? (warps >= 4 ? append_bounds_kernel<128, 4> : warps == 2 ? append_bounds_kernel<128, 2> : append_bounds_kernel<128, 1>)
                                  : (warps >= 4 ? append_bounds_kernel<64, 4> : warps == 2 ? append_bounds_kernel<64, 2> : append_bounds_kernel<64, 1>);
    e = launch_kernel(kern, grid, dim3(kThreads), 0, stream, p);
  } else {
    const int64_t per = kBatch * (kThreads / (a->cache.D / 8)), rows = a->T * a->B * a->cache.Hkv;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>((rows + per - 1) / per, static_cast<int64_t>(num_sms()) * 16)));
    e = a->cache.D == 128 ? launch_kernel(append_rows_kernel<128>, grid, dim3(kThreads), 0, stream, p)
                          : launch_kernel(append_rows_kernel<64>, grid, dim3(kThreads), 0, stream, p);
  }
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged append launch");
  return BSA_OK;
}

}  // namespace bsa
