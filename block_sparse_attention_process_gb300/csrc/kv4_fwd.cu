// Attention of new tokens over the 4-bit cache: o = sum_j p_j v_j, p_j =
// exp(s_j - lse), s_j = scale q.k_j (capped), over the slots a token sees.
//
// One CTA per (sequence, q head, new token): scores into the workspace, the
// softmax statistics by a block reduction, then one output element per
// thread.  A second kernel adds the probabilities of a key's rows to its
// accumulated weight.
#include <cmath>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

struct Kv4FwdParams {
  bsa_kv4_cache c;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int64_t qs[3], os[3];
  int32_t Hq, T, G;
  const int32_t *lens, *q_lens;
  float scale, cap;
  const float* sinks;
  int32_t n_sinks, sinks_kv;
  int32_t accumulate;
  float* scores;  // [B, Hq, T, capacity]
  uint32_t* err;
};

// Slots that token t of sequence b sees: [0, end).
__device__ __forceinline__ int32_t visible_end(const Kv4FwdParams& p, int32_t b, int32_t t, uint32_t* err) {
  const int32_t len = clamp_len(p.lens[b], p.c.capacity, err);
  const int32_t n = p.q_lens ? min(max(p.q_lens[b], 0), p.T) : p.T;
  if (t >= n) return 0;
  return max(0, len - n + t + 1);
}

template <int D>
__global__ void __launch_bounds__(256) fwd_rows_kernel(const __grid_constant__ Kv4FwdParams p) {
  __shared__ float q[D], red[8], part[256];
  griddep_launch_dependents();
  griddep_wait();
  const int32_t row = static_cast<int32_t>(blockIdx.x);
  const int32_t t = row % p.T, hq = row / p.T % p.Hq, b = row / p.T / p.Hq;
  const int32_t h = hq / p.G;
  const int64_t head = (static_cast<int64_t>(b) * p.c.Hkv + h) * p.c.capacity;
  if (threadIdx.x < D) q[threadIdx.x] = __bfloat162float(p.q[b * p.qs[0] + hq * p.qs[1] + t * p.qs[2] + threadIdx.x]);
  __syncthreads();
  const int32_t end = visible_end(p, b, t, threadIdx.x == 0 ? p.err : nullptr);
  float* x = p.scores + static_cast<int64_t>(row) * p.c.capacity;
  float m = -INFINITY;
  for (int32_t j = threadIdx.x; j < end; j += 256) {
    float s = 0.f;
    for (int w = 0; w < Kv4<D>::kWords; ++w) {
      const uint32_t c = static_cast<const uint32_t*>(p.c.k_codes)[(head + j) * Kv4<D>::kWords + w];
      float dot = 0.f;
      for (int i = 0; i < 8; ++i)
        dot = fmaf(static_cast<float>(static_cast<int>((c >> (4 * i)) & 15u) - 8), q[k_word_elem<D>(w) + i], dot);
      s = fmaf(dot, __bfloat162float(static_cast<const __nv_bfloat16*>(p.c.k_scales)[(head + j) * Kv4<D>::kGroups + w % Kv4<D>::kGroups]), s);
    }
    s *= p.scale;
    if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
    x[j] = s;
    m = fmaxf(m, s);
  }
  for (int32_t j = threadIdx.x; j < p.n_sinks; j += 256) m = fmaxf(m, p.sinks[(p.sinks_kv ? h * p.n_sinks : 0) + j]);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = m;
  __syncthreads();
  for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
  __syncthreads();
  float l = 0.f;
  for (int32_t j = threadIdx.x; j < end; j += 256) l += expf(x[j] - m);
  for (int32_t j = threadIdx.x; j < p.n_sinks; j += 256) l += expf(p.sinks[(p.sinks_kv ? h * p.n_sinks : 0) + j] - m);
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = l;
  __syncthreads();
  l = 0.f;
  for (int i = 0; i < 8; ++i) l += red[i];
  const float lse = l > 0.f ? m + logf(l) : (m == -INFINITY ? -INFINITY : NAN);
  if (threadIdx.x == 0) p.lse[row] = lse;
  // output element d: 256 / D threads share it
  const int d = threadIdx.x % D;
  const int g = d / 32, word = (d % 32 / 4) * Kv4<D>::kGroups + g;
  float acc = 0.f;
  for (int32_t j = threadIdx.x / D; j < end; j += 256 / D) {
    const uint32_t c = static_cast<const uint16_t*>(p.c.v_codes)[(head + j) * 2 * Kv4<D>::kWords + (word ^ (2 * v_word_swap<D>(j)))];
    const float s = __bfloat162float(static_cast<const __nv_bfloat16*>(p.c.v_scales)[(head + j) * Kv4<D>::kGroups + g]);
    acc = fmaf(expf(x[j] - lse), s * static_cast<float>(static_cast<int>((c >> (4 * (d % 4))) & 15u) - 8), acc);
  }
  part[threadIdx.x] = acc;
  __syncthreads();
  if (threadIdx.x < D) {
    for (int i = 1; i < 256 / D; ++i) acc += part[threadIdx.x + i * D];
    p.o[b * p.os[0] + hq * p.os[1] + t * p.os[2] + d] = __float2bfloat16_rn(acc);
  }
}

__global__ void __launch_bounds__(256) fwd_weights_kernel(const __grid_constant__ Kv4FwdParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int32_t bh = static_cast<int32_t>(blockIdx.y), b = bh / p.c.Hkv, h = bh % p.c.Hkv;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= p.c.capacity) return;
  float w = 0.f;
  for (int32_t r = 0; r < p.G * p.T; ++r) {
    const int32_t t = r % p.T, hq = h * p.G + r / p.T;
    if (j >= visible_end(p, b, t, nullptr)) continue;
    const int64_t row = (static_cast<int64_t>(b) * p.Hq + hq) * p.T + t;
    w += expf(p.scores[row * p.c.capacity + j] - p.lse[row]);
  }
  p.c.weights[bh * p.c.capacity + j] += w;
}

}  // namespace

size_t kv4_fwd_workspace_bytes(const bsa_kv4_fwd_args* a) {
  return static_cast<size_t>(a->cache.B) * a->Hq * a->T * a->cache.capacity * sizeof(float);
}

bsa_status kv4_fwd_launch(const bsa_kv4_fwd_args* a, float scale, cudaStream_t stream) {
  Kv4FwdParams p{};
  p.c = a->cache;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.o = static_cast<__nv_bfloat16*>(a->o);
  p.lse = a->lse;
  for (int i = 0; i < 3; ++i) {
    p.qs[i] = a->q_stride[i];
    p.os[i] = a->o_stride[i];
  }
  p.Hq = a->Hq;
  p.T = static_cast<int32_t>(a->T);
  p.G = a->Hq / a->cache.Hkv;
  p.lens = a->lens;
  p.q_lens = a->q_lens;
  p.scale = scale;
  p.cap = a->logits_soft_cap;
  p.sinks = a->sinks;
  p.n_sinks = a->num_sinks;
  p.sinks_kv = a->sinks_per_kv_head ? 1 : 0;
  p.accumulate = a->accumulate;
  p.scores = static_cast<float*>(a->workspace);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  const unsigned rows = static_cast<unsigned>(a->cache.B) * a->Hq * static_cast<unsigned>(a->T);
  cudaError_t e = a->cache.D == 128 ? launch_kernel(fwd_rows_kernel<128>, dim3(rows), dim3(256), 0, stream, p)
                                    : launch_kernel(fwd_rows_kernel<64>, dim3(rows), dim3(256), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "kv4 forward launch");
  if (a->accumulate) {
    e = launch_kernel(fwd_weights_kernel, dim3(static_cast<unsigned>((a->cache.capacity + 255) / 256), a->cache.B * a->cache.Hkv),
                      dim3(256), 0, stream, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "kv4 weights launch");
  }
  return BSA_OK;
}

}  // namespace bsa
