// Quantisation of new keys and values into the 4-bit cache.
//
// Per group of 32 elements: s = bf16(max|x| / 7), c = rint(x / s) + 8.  The
// quotient is x (1/s) and one correction: x has 8 significant bits and s/2 times
// an odd number at most 12, so a quotient that is not itself a tie is at least
// 2^-15 (relative) away from one and rounds right, and a tie, a number of few
// bits, comes out exactly.
//
// HBM-bound: 4 D bytes read and D + D/8 of codes and scales (+ 4 D of values)
// written per token and head.  A row takes D/8 lanes: for K each lane holds
// 8 consecutive elements, which are one 4-byte word of codes; for V its two
// quads of elements 32 apart, likewise one word.  4 x 8 x 8192 rows of 128 with
// their values take 63 us, 72% of the copy bandwidth, and 58 without values, 44% of
// it.  The rest is instructions (68% of the issue slots) and latency:
// 98 us with a true division per element, 72 with ties found by their remainder
// and maxima one element at a time.  One row a lane: two in flight measured
// slower (fewer warps fit).
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

// Division of numbers below 2^31 by one known on the host.
struct Divisor {
  uint32_t d, mul, shift;
  Divisor() = default;
  explicit Divisor(uint32_t n) : d(n), mul(0), shift(0) {
    while ((uint64_t(1) << shift) < n) ++shift;
    mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - n)) / n + 1);
  }
};
__device__ __forceinline__ uint32_t quotient(uint32_t x, const Divisor& v) { return (__umulhi(x, v.mul) + x) >> v.shift; }

struct AppendParams {
  bsa_kv4_cache c;
  const __nv_bfloat16 *k, *v;
  int64_t ks[3], vs[3];
  uint32_t T, rows;
  Divisor by_t, by_h;
  const int32_t *start, *n_new, *first_position;
  const float* weights0;
  __nv_bfloat16 *k_values, *v_values;
  uint32_t* err;
};

__device__ __forceinline__ float rcp_approx(float x) {  // off by 2^-23 at most
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest magnitudes of the two halves as bf16 bits (NaN above infinity above every number).
__device__ __forceinline__ uint32_t max_bits(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7FFF7FFFu); }

// The group's scale (bf16 bits) from its largest magnitude.
__device__ __forceinline__ uint32_t scale_bits(uint32_t m) {
  if (m >= 0x7F80u) return 0x7FC0u;  // an infinity or a NaN in the group: it reads as NaN
  // (times 1/7: a seventh of a bf16 number is no midpoint of two bf16 numbers, nor within 2^-12 of one)
  const __nv_bfloat16 s = __float2bfloat16_rn(__uint_as_float(m << 16) * (1.0f / 7.0f));
  return static_cast<uint32_t>(__bfloat16_as_ushort(s));
}

// q = rint(x / s), |q| <= 7.  One step of Newton's method: a quotient that is a
// tie comes out exactly, any other is at least 2^-15 (relative) away from one.
__device__ __forceinline__ float quantise(float x, float s, float inv) {
  constexpr float kMagic = 12582912.f;  // 1.5 2^23: the sum is rounded to a whole number, ties to even
  const float q = x * inv;
  return fmaf(fmaf(-q, s, x), inv, q) + kMagic - kMagic;
}
// The same by a true division, for scales that are 0, NaN or so small that
// their reciprocal might overflow.
__device__ __forceinline__ float quantise_slow(float x, float s) {
  // (a subnormal scale is coarse: the largest elements may be 7.5 of it and more)
  return s > 0.f ? fminf(fmaxf(rintf(x / s), -7.f), 7.f) : 0.f;
}

// Four bf16 elements (two words) -> four codes in the low 16 bits; the values
// they stand for replace the elements.
template <bool kSlow>
__device__ __forceinline__ uint32_t quantise4(uint32_t& w0, uint32_t& w1, float s, float inv) {
  float x[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)}, q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = kSlow ? quantise_slow(x[i], s) : quantise(x[i], s, inv);
  w0 = pack_bf16x2(q[0] * s, q[1] * s);
  w1 = pack_bf16x2(q[2] * s, q[3] * s);
  // the four codes as one whole number, exact in fp32, in the last bits of a sum with 2^23
  return __float_as_uint(fmaf(q[3], 4096.f, fmaf(q[2], 256.f, fmaf(q[1], 16.f, q[0]))) + (8388608.f + 0x8888)) & 0xFFFFu;
}

// A lane's eight elements of K and two quads of V (bits of their scales): the
// codes of both, the values in the elements' place.
template <bool kSlow>
__device__ __forceinline__ uint2 quantise_lane(uint4& k, uint2& va, uint2& vb, uint32_t sk, uint32_t sa, uint32_t sb) {
  const float fk = __uint_as_float(sk << 16), fa = __uint_as_float(sa << 16), fb = __uint_as_float(sb << 16);
  const float ik = rcp_approx(fk), ia = rcp_approx(fa), ib = rcp_approx(fb);  // (slow: not used)
  uint2 c;
  c.x = quantise4<kSlow>(k.x, k.y, fk, ik) | quantise4<kSlow>(k.z, k.w, fk, ik) << 16;
  c.y = quantise4<kSlow>(va.x, va.y, fa, ia) | quantise4<kSlow>(vb.x, vb.y, fb, ib) << 16;
  return c;
}

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = Kv4<D>::kWords;  // lanes of one row
  constexpr int kPiece = Kv4<D>::kPieceWords;
  constexpr uint32_t kRowsCta = 256 / kLanes;
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t u = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int d0 = v_word_elem<D>(u, 0), d1 = v_word_elem<D>(u, 1);
  // rows (b, h, t) in order (every lane of a warp makes the same number of trips: the shuffles)
  for (uint64_t r0 = static_cast<uint64_t>(blockIdx.x) * kRowsCta; r0 < p.rows; r0 += static_cast<uint64_t>(gridDim.x) * kRowsCta) {
    const uint64_t row = r0 + sub;
    const bool in = row < p.rows;
    const uint32_t bh = in ? quotient(static_cast<uint32_t>(row), p.by_t) : 0;
    const uint32_t t = in ? static_cast<uint32_t>(row) - bh * p.T : 0;
    const uint32_t b = quotient(bh, p.by_h), h = bh - b * static_cast<uint32_t>(p.c.Hkv);
    const bool fresh = in && (!p.n_new || static_cast<int32_t>(t) < p.n_new[b]);
    uint4 kw = make_uint4(0, 0, 0, 0);
    uint2 va = make_uint2(0, 0), vb = make_uint2(0, 0);
    if (fresh) {
      const __nv_bfloat16* vr = p.v + b * p.vs[0] + h * p.vs[1] + t * p.vs[2];
      kw = __ldcs(reinterpret_cast<const uint4*>(p.k + b * p.ks[0] + h * p.ks[1] + t * p.ks[2] + 8 * u));
      va = __ldcs(reinterpret_cast<const uint2*>(vr + d0));
      vb = __ldcs(reinterpret_cast<const uint2*>(vr + d1));
    }
    // a K group is 4 neighbouring lanes, a V group every kPiece-th lane of the row
    const uint32_t m2 = max_bits(max_bits(max_bits(kw.x & 0x7FFF7FFFu, kw.y), kw.z), kw.w);
    const uint32_t ma = max_bits(va.x & 0x7FFF7FFFu, va.y), mb = max_bits(vb.x & 0x7FFF7FFFu, vb.y);
    uint32_t mk = max(m2 & 0xFFFFu, m2 >> 16);
    uint32_t mv = __vmaxu2(__byte_perm(ma, mb, 0x5410), __byte_perm(ma, mb, 0x7632));
#pragma unroll
    for (int o = 1; o < 4; o *= 2) mk = max(mk, __shfl_xor_sync(0xffffffffu, mk, o));
#pragma unroll
    for (int o = kPiece; o < 8 * kPiece; o *= 2) mv = __vmaxu2(mv, __shfl_xor_sync(0xffffffffu, mv, o));
    const uint32_t sk = scale_bits(mk), sa = scale_bits(mv & 0xFFFFu), sb = scale_bits(mv >> 16);
    // 2^-100 <= s, and not NaN
    constexpr uint32_t kLeast = (127u - 100u) << 7, kSpan = 0x7F80u - kLeast;
    const bool usual = max(max(sk - kLeast, sa - kLeast), sb - kLeast) < kSpan;
    const uint2 c = __all_sync(0xffffffffu, usual) ? quantise_lane<false>(kw, va, vb, sk, sa, sb)
                                                   : quantise_lane<true>(kw, va, vb, sk, sa, sb);
    if (fresh) {
      const int64_t slot = static_cast<int64_t>(p.start[b]) + t;
      if (slot >= 0 && slot < p.c.capacity) {
        const int64_t at = bh * p.c.capacity + slot;
        // elements 8 u + 0..7 of K are group u / 4, piece u % 4
        static_cast<uint32_t*>(p.c.k_codes)[at * kLanes + (u % 4) * Kv4<D>::kGroups + u / 4] = c.x;
        static_cast<uint32_t*>(p.c.v_codes)[at * kLanes + (u ^ v_word_swap<D>(slot))] = c.y;
        if (u % 4 == 0) static_cast<uint16_t*>(p.c.k_scales)[at * Kv4<D>::kGroups + u / 4] = static_cast<uint16_t>(sk);
        if (u < kPiece) static_cast<uint32_t*>(p.c.v_scales)[at * kPiece + u] = sa | (sb << 16);
        if (u == 0 && p.c.weights) p.c.weights[at] = p.weights0 ? p.weights0[row] : 0.f;
        if (u == 1 && p.c.positions)
          p.c.positions[at] = (p.first_position ? p.first_position[b] : p.start[b]) + static_cast<int32_t>(t);
      } else if (u == 0 && p.err) {
        atomicOr(p.err, DEV_ERR_BOUNDS);
      }
    }
    // (padding rows: the elements are 0 and so are their values)
    if (in && p.k_values) __stcs(reinterpret_cast<uint4*>(p.k_values + row * D + 8 * u), kw);
    if (in && p.v_values) {
      __stcs(reinterpret_cast<uint2*>(p.v_values + row * D + d0), va);
      __stcs(reinterpret_cast<uint2*>(p.v_values + row * D + d1), vb);
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
  p.T = static_cast<uint32_t>(a->T);
  p.rows = static_cast<uint32_t>(a->cache.B) * a->cache.Hkv * p.T;
  p.by_t = Divisor(p.T);
  p.by_h = Divisor(static_cast<uint32_t>(a->cache.Hkv));
  p.start = a->start;
  p.n_new = a->n_new;
  p.first_position = a->first_position;
  p.weights0 = a->weights0;
  p.k_values = static_cast<__nv_bfloat16*>(a->k_values);
  p.v_values = static_cast<__nv_bfloat16*>(a->v_values);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  const int64_t per = 256 / (a->cache.D / 8);
  const int grid = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(p.rows) + per - 1) / per, static_cast<int64_t>(num_sms()) * 16));
  cudaError_t e = a->cache.D == 128 ? launch_kernel(append_kernel<128>, dim3(grid), dim3(256), 0, stream, p)
                                    : launch_kernel(append_kernel<64>, dim3(grid), dim3(256), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 append launch");
  return BSA_OK;
}

}  // namespace bsa
