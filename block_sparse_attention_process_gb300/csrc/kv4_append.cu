// Quantisation of new keys and values into the 4-bit cache.
//
// Per group of 32 elements: s = bf16(max|x| / 7), c = rint(x / s) + 8.  The
// fp32 quotient rounds to the same integer as the exact one: x has 8
// significant bits and s/2 times an odd number at most 12, so a quotient that
// is not itself a tie is at least 2^-15 (relative) away from one.
//
// HBM-bound: 4 D bytes read and D + D/4 codes and scales (+ 4 D values)
// written per token and head.  A row takes D/8 lanes: for K each lane holds
// 8 consecutive elements, which are one 4-byte word of codes; for V its two
// quads of elements 32 apart, likewise one word.
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

struct AppendParams {
  bsa_kv4_cache c;
  const __nv_bfloat16 *k, *v;
  int64_t ks[3], vs[3];
  int64_t T, rows;
  const int32_t *start, *n_new, *first_position;
  const float* weights0;
  __nv_bfloat16 *k_values, *v_values;
  uint32_t* err;
};

// Largest magnitude as bf16 bits (NaN above infinity above every number).
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t w) {
  m = max(m, w & 0x7FFFu);
  return max(m, (w >> 16) & 0x7FFFu);
}

// The group's scale (bf16 bits) from its largest magnitude.
__device__ __forceinline__ uint32_t scale_bits(uint32_t m) {
  if (m >= 0x7F80u) return 0x7FC0u;  // an infinity or a NaN in the group: it reads as NaN
  const __nv_bfloat16 s = __float2bfloat16_rn(__uint_as_float(m << 16) / 7.0f);
  return static_cast<uint32_t>(__bfloat16_as_ushort(s));
}

// Four bf16 elements (two words) -> four codes in the low 16 bits; the values
// they stand for replace the elements.
__device__ __forceinline__ uint32_t quantise4(uint32_t& w0, uint32_t& w1, uint32_t sbits) {
  const float s = __uint_as_float(sbits << 16);
  float x[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)};
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float q = s > 0.f ? rintf(x[i] / s) : 0.f;
    c |= static_cast<uint32_t>(static_cast<int>(q) + 8) << (4 * i);
    x[i] = q * s;
  }
  w0 = pack_bf16x2(x[0], x[1]);
  w1 = pack_bf16x2(x[2], x[3]);
  return c;
}

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = Kv4<D>::kWords;  // lanes of one row
  constexpr int kPiece = Kv4<D>::kPieceWords;
  griddep_launch_dependents();
  griddep_wait();
  const int u = threadIdx.x % kLanes;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (256 / kLanes);
  // every lane of a warp makes the same number of trips (the shuffles)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * (256 / kLanes); r0 < p.rows; r0 += step) {
    const int64_t row = r0 + threadIdx.x / kLanes;
    const bool in = row < p.rows;
    const int64_t t = in ? row % p.T : 0, bh = in ? row / p.T : 0;
    const int64_t b = bh / p.c.Hkv, h = bh % p.c.Hkv;
    const bool fresh = in && (!p.n_new || t < p.n_new[b]);
    const int64_t slot = fresh ? static_cast<int64_t>(p.start[b]) + t : 0;
    const bool fits = slot >= 0 && slot < p.c.capacity;
    if (fresh && !fits && u == 0 && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
    uint4 kw = make_uint4(0, 0, 0, 0);
    uint2 va = make_uint2(0, 0), vb = make_uint2(0, 0);
    const int d0 = v_word_elem<D>(u, 0), d1 = v_word_elem<D>(u, 1);
    if (fresh) {
      kw = *reinterpret_cast<const uint4*>(p.k + b * p.ks[0] + h * p.ks[1] + t * p.ks[2] + 8 * u);
      const __nv_bfloat16* vrow = p.v + b * p.vs[0] + h * p.vs[1] + t * p.vs[2];
      va = *reinterpret_cast<const uint2*>(vrow + d0);
      vb = *reinterpret_cast<const uint2*>(vrow + d1);
    }
    // a K group is 4 neighbouring lanes, a V group every kPiece-th lane of the row
    uint32_t mk = max_bits(max_bits(max_bits(max_bits(0, kw.x), kw.y), kw.z), kw.w);
    uint32_t ma = max_bits(max_bits(0, va.x), va.y), mb = max_bits(max_bits(0, vb.x), vb.y);
#pragma unroll
    for (int o = 1; o < 4; o *= 2) mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
#pragma unroll
    for (int o = kPiece; o < 8 * kPiece; o *= 2) {
      ma = max(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    const uint32_t sk = scale_bits(mk), sa = scale_bits(ma), sb = scale_bits(mb);
    const uint32_t ck = quantise4(kw.x, kw.y, sk) | (quantise4(kw.z, kw.w, sk) << 16);
    const uint32_t cv = quantise4(va.x, va.y, sa) | (quantise4(vb.x, vb.y, sb) << 16);
    if (fresh && fits) {
      const int64_t at = (b * p.c.Hkv + h) * p.c.capacity + slot;
      // elements 8 u + 0..7 of K are group u / 4, piece u % 4
      static_cast<uint32_t*>(p.c.k_codes)[at * kLanes + (u % 4) * Kv4<D>::kGroups + u / 4] = ck;
      static_cast<uint32_t*>(p.c.v_codes)[at * kLanes + (u ^ v_word_swap<D>(slot))] = cv;
      if (u % 4 == 0) static_cast<uint16_t*>(p.c.k_scales)[at * Kv4<D>::kGroups + u / 4] = static_cast<uint16_t>(sk);
      if (u < kPiece) static_cast<uint32_t*>(p.c.v_scales)[at * kPiece + u] = sa | (sb << 16);
      if (u == 0 && p.c.weights) p.c.weights[at] = p.weights0 ? p.weights0[row] : 0.f;
      if (u == 0 && p.c.positions)
        p.c.positions[at] = (p.first_position ? p.first_position[b] : p.start[b]) + static_cast<int32_t>(t);
    }
    // (padding rows: the elements are 0 and so are their values)
    if (in && p.k_values) *reinterpret_cast<uint4*>(p.k_values + row * D + 8 * u) = kw;
    if (in && p.v_values) {
      *reinterpret_cast<uint2*>(p.v_values + row * D + d0) = va;
      *reinterpret_cast<uint2*>(p.v_values + row * D + d1) = vb;
    }
  }
}

}  // namespace

bsa_status kv4_append_launch(const bsa_kv4_append_args* a, cudaStream_t stream) {
  AppendParams p{};
  p.c = a->cache;
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.v = static_cast<const __nv_bfloat16*>(a->v);
  for (int i = 0; i < 3; ++i) {
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
  }
  p.T = a->T;
  p.rows = static_cast<int64_t>(a->cache.B) * a->cache.Hkv * a->T;
  p.start = a->start;
  p.n_new = a->n_new;
  p.first_position = a->first_position;
  p.weights0 = a->weights0;
  p.k_values = static_cast<__nv_bfloat16*>(a->k_values);
  p.v_values = static_cast<__nv_bfloat16*>(a->v_values);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  const int per = 256 / (a->cache.D / 8);
  const int grid = static_cast<int>(std::min<int64_t>((p.rows + per - 1) / per, static_cast<int64_t>(num_sms()) * 16));
  cudaError_t e = a->cache.D == 128 ? launch_kernel(append_kernel<128>, dim3(grid), dim3(256), 0, stream, p)
                                    : launch_kernel(append_kernel<64>, dim3(grid), dim3(256), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 append launch");
  return BSA_OK;
}

}  // namespace bsa
