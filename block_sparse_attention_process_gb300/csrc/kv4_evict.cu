// Eviction from the 4-bit cache by accumulated attention weight.
//
// Per (sequence, key head): the `keep` slots of the largest key, key = the
// weight as an ordered 32-bit integer (recent tokens above everything, NaN
// above every number), ties to the lower slot.  A radix select of four 8-bit
// digits finds the smallest kept key; one ordered pass then writes for every
// kept slot where it goes, and a second kernel moves the rows.
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

constexpr int kSelThreads = 1024;

struct EvictParams {
  bsa_kv4_cache c, o;
  const int32_t *lens, *seen;
  int64_t keep, recent;
  int32_t in_place;
  int32_t* new_lens;
  int32_t* index;
  __nv_bfloat16 *k_values, *v_values;
  int32_t* holes;  // workspace [B, Hkv, keep] (in place only)
  uint32_t* err;
};

// Weights as unsigned integers in increasing order.
__device__ __forceinline__ uint32_t order_key(float w, bool recent) {
  if (recent) return 0xFFFFFFFFu;
  if (isnan(w)) return 0xFFFFFFFEu;
  const uint32_t u = __float_as_uint(w + 0.0f);  // (-0 and 0 are equal)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the CTA of one 0/1 flag per thread, and the total.
__device__ __forceinline__ int32_t block_rank(bool flag, int32_t* warp_sums, int32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t votes = __ballot_sync(0xffffffffu, flag);
  __syncthreads();  // the sums of the call before have been read
  if (lane == 0) warp_sums[warp] = __popc(votes);
  __syncthreads();
  int32_t before = 0, all = 0;
  const int32_t mine = lane < kSelThreads / 32 ? warp_sums[lane] : 0;
  int32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  before = __shfl_sync(0xffffffffu, inc - mine, warp);
  all = __shfl_sync(0xffffffffu, inc, 31);
  total = all;
  return before + __popc(votes & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ int32_t warp_sums[32];
  __shared__ uint32_t pick[2];
  griddep_launch_dependents();
  griddep_wait();
  const int64_t bh = blockIdx.x;
  const int32_t b = static_cast<int32_t>(bh / p.c.Hkv);
  const int32_t n = clamp_len(p.lens[b], p.c.capacity, threadIdx.x == 0 ? p.err : nullptr);
  const int64_t first_recent = static_cast<int64_t>(p.seen ? p.seen[b] : p.lens[b]) - p.recent;
  const float* w = p.c.weights + bh * p.c.capacity;
  const int32_t* pos = p.c.positions ? p.c.positions + bh * p.c.capacity : nullptr;
  int32_t* index = p.index + bh * p.keep;
  const int32_t keep = static_cast<int32_t>(p.keep < n ? p.keep : n);
  if (threadIdx.x == 0 && bh % p.c.Hkv == 0) p.new_lens[b] = keep;
  auto key_of = [&](int32_t i) {
    const bool recent = p.recent > 0 && (pos ? static_cast<int64_t>(pos[i]) : i) >= first_recent;
    return order_key(w[i], recent);
  };

  uint32_t least = 0;      // smallest kept key
  int32_t ties = n;        // how many slots with that key are kept
  if (n > p.keep) {
    uint32_t prefix = 0, mask = 0;
    uint32_t want = static_cast<uint32_t>(p.keep);  // rank (1-based, from the top) among keys with this prefix
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int32_t i = threadIdx.x; i < n; i += kSelThreads) {
        const uint32_t k = key_of(i);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t above = 0;
        int d = 255;
        while (d > 0 && above + hist[d] < want) above += hist[d--];
        pick[0] = static_cast<uint32_t>(d);
        pick[1] = want - above;
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= 255u << shift;
      want = pick[1];
      __syncthreads();
    }
    least = prefix;
    ties = static_cast<int32_t>(want);
  }

  // one ordered pass: which slots stay, and where their tokens go
  int32_t kept_before = 0, ties_before = 0, holes_before = 0;
  for (int32_t i0 = 0; i0 < n; i0 += kSelThreads) {
    const int32_t i = i0 + static_cast<int32_t>(threadIdx.x);
    const uint32_t k = i < n ? key_of(i) : 0u;
    int32_t total;
    const bool tie = i < n && k == least && n > p.keep;
    const int32_t tr = block_rank(tie, warp_sums, total) + ties_before;
    ties_before += total;
    const bool stay = i < n && (n <= p.keep || k > least || (tie && tr < ties));
    if (!p.in_place) {
      const int32_t r = block_rank(stay, warp_sums, total) + kept_before;
      kept_before += total;
      if (stay) index[r] = i;
    } else {
      const bool hole = i < n && i < p.keep && !stay;
      const int32_t hr = block_rank(hole, warp_sums, total) + holes_before;
      holes_before += total;
      if (hole) p.holes[bh * p.keep + hr] = i;
      if (stay && i < p.keep) index[i] = i;
      const bool mover = stay && i >= p.keep;
      // (the holes all lie below slot keep, so a mover's hole is already written:
      // by this trip or an earlier one, and block_rank has barriers in between)
      const int32_t mr = block_rank(mover, warp_sums, total) + kept_before;
      kept_before += total;
      if (mover) index[p.holes[bh * p.keep + mr]] = i;
    }
  }
  for (int64_t r = keep + static_cast<int64_t>(threadIdx.x); r < p.keep; r += kSelThreads) index[r] = -1;
}

__device__ __forceinline__ float code_value(uint32_t w, int i, float s) {
  return static_cast<float>(static_cast<int>((w >> (4 * i)) & 15u) - 8) * s;
}

template <int D>
__global__ void __launch_bounds__(256) move_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kLanes = Kv4<D>::kWords;
  constexpr int kPiece = Kv4<D>::kPieceWords;
  constexpr int kGroups = Kv4<D>::kGroups;
  griddep_launch_dependents();
  griddep_wait();
  const int u = threadIdx.x % kLanes;
  const int64_t rows = static_cast<int64_t>(p.c.B) * p.c.Hkv * p.keep;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (256 / kLanes);
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes; row < rows; row += step) {
    const int64_t bh = row / p.keep, r = row % p.keep;
    const int32_t src = p.index[row];
    const bool live = src >= 0;
    if (!live && !p.k_values && !p.v_values) continue;
    uint32_t kw = 0x88888888u, vw = 0x88888888u, ks = 0, vs = 0;
    if (live) {
      const int64_t from = bh * p.c.capacity + src, to = bh * p.o.capacity + r;
      kw = static_cast<const uint32_t*>(p.c.k_codes)[from * kLanes + u];
      vw = static_cast<const uint32_t*>(p.c.v_codes)[from * kLanes + (u ^ v_word_swap<D>(src))];
      ks = static_cast<const uint16_t*>(p.c.k_scales)[from * kGroups + u % kGroups];
      vs = static_cast<const uint32_t*>(p.c.v_scales)[from * kPiece + u % kPiece];
      if (!p.in_place || src != r) {
        static_cast<uint32_t*>(p.o.k_codes)[to * kLanes + u] = kw;
        static_cast<uint32_t*>(p.o.v_codes)[to * kLanes + (u ^ v_word_swap<D>(r))] = vw;
        if (u < kGroups) static_cast<uint16_t*>(p.o.k_scales)[to * kGroups + u] = static_cast<uint16_t>(ks);
        if (u < kPiece) static_cast<uint32_t*>(p.o.v_scales)[to * kPiece + u] = vs;
        if (u == 0 && p.o.weights) p.o.weights[to] = p.c.weights[from];
        if (u == 1 && p.o.positions)
          p.o.positions[to] = p.c.positions ? p.c.positions[from] : src;
      }
    }
    if (p.k_values) {
      const float s = __uint_as_float(ks << 16);
      uint4 o;
      o.x = pack_bf16x2(code_value(kw, 0, s), code_value(kw, 1, s));
      o.y = pack_bf16x2(code_value(kw, 2, s), code_value(kw, 3, s));
      o.z = pack_bf16x2(code_value(kw, 4, s), code_value(kw, 5, s));
      o.w = pack_bf16x2(code_value(kw, 6, s), code_value(kw, 7, s));
      *reinterpret_cast<uint4*>(p.k_values + row * D + k_word_elem<D>(u)) = o;
    }
    if (p.v_values) {
      const float s0 = bf16_lo(vs), s1 = bf16_hi(vs);
      *reinterpret_cast<uint2*>(p.v_values + row * D + v_word_elem<D>(u, 0)) =
          make_uint2(pack_bf16x2(code_value(vw, 0, s0), code_value(vw, 1, s0)),
                     pack_bf16x2(code_value(vw, 2, s0), code_value(vw, 3, s0)));
      *reinterpret_cast<uint2*>(p.v_values + row * D + v_word_elem<D>(u, 1)) =
          make_uint2(pack_bf16x2(code_value(vw, 4, s1), code_value(vw, 5, s1)),
                     pack_bf16x2(code_value(vw, 6, s1), code_value(vw, 7, s1)));
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
  cudaError_t e = launch_kernel(select_kernel, dim3(a->cache.B * a->cache.Hkv), dim3(kSelThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 evict selection launch");
  const int64_t rows = static_cast<int64_t>(a->cache.B) * a->cache.Hkv * a->keep;
  const int per = 256 / (a->cache.D / 8);
  const int grid = static_cast<int>(std::min<int64_t>((rows + per - 1) / per, static_cast<int64_t>(num_sms()) * 16));
  e = a->cache.D == 128 ? launch_kernel(move_kernel<128>, dim3(grid), dim3(256), 0, stream, p)
                        : launch_kernel(move_kernel<64>, dim3(grid), dim3(256), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 evict move launch");
  return BSA_OK;
}

}  // namespace bsa
