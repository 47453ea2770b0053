// The attention weight every key of a prompt has received:
//   w[j] = sum over the group's q heads and the queries i that see j of exp(scale q_i.k_j - lse_i).
// The loop is the dK/dV launch's: a tile is a key block, its items the
// non-empty query blocks of each q head's row of the dkv MaskInfo.
//
// One CTA per tile, one key per thread, the item's queries through shared
// memory.
#include <cmath>

#include "internal.h"
#include "maskinfo_dev.cuh"
#include "ptx.cuh"

namespace bsa {
namespace {

struct KeyWeightsParams {
  const __nv_bfloat16 *q, *k;
  const float* lse;
  const int32_t* q_lens;
  float* out;
  int32_t B, Hq, Hkv, nK;
  int64_t Sq, Skv;
  float scale, cap;
  MaskInfoDev mi;
  uint32_t* err;
};

template <int D>
__global__ void __launch_bounds__(128) key_weights_kernel(const __grid_constant__ KeyWeightsParams p) {
  __shared__ float qs[32][D];
  griddep_launch_dependents();
  griddep_wait();
  const int32_t j = static_cast<int32_t>(blockIdx.x), g = static_cast<int32_t>(blockIdx.y), b = static_cast<int32_t>(blockIdx.z);
  const int32_t G = p.Hq / p.Hkv;
  const int64_t key = static_cast<int64_t>(j) * 128 + threadIdx.x;
  float kv[D];
  const __nv_bfloat16* krow = p.k + ((static_cast<int64_t>(b) * p.Hkv + g) * p.Skv + key) * D;
#pragma unroll
  for (int d = 0; d < D; ++d) kv[d] = __bfloat162float(krow[d]);
  int64_t lo, hi;
  query_interval(p.mi.kind, p.mi.left, p.mi.right, p.mi.chunk, key, lo, hi);
  const int64_t q_end = p.q_lens ? p.q_lens[b] : p.Sq;
  float w = 0.f;
  for (int32_t gh = 0; gh < G; ++gh) {
    const int32_t hq = g * G + gh, hm = p.mi.heads == 1 ? 0 : hq;
    const int64_t row_base = (static_cast<int64_t>(hm) * p.mi.rows + j) * p.mi.width;
    const int64_t head = (static_cast<int64_t>(b) * p.Hq + hq) * p.Sq;
    for (int32_t t = 0; t < p.mi.width; ++t) {
      const BlockRef br = read_block(p.mi, row_base, t, threadIdx.x == 0 ? p.err : nullptr);
      if (br.label == 0) continue;
      for (int32_t i0 = 0; i0 < 128; i0 += 32) {
        __syncthreads();
        for (int x = threadIdx.x; x < 32 * D; x += 128)
          qs[x / D][x % D] = __bfloat162float(p.q[(head + br.col * 128 + i0 + x / D) * D + x % D]);
        __syncthreads();
        for (int32_t i = 0; i < 32; ++i) {
          const int64_t qi = static_cast<int64_t>(br.col) * 128 + i0 + i;
          const float lse = p.lse[head + qi];
          bool seen = qi < q_end && lse != -INFINITY;
          if (br.label == 1)
            seen = seen && (p.mi.kind == BSA_MASK_DENSE
                                ? p.mi.partial[(static_cast<int64_t>(br.slot) * 128 + threadIdx.x) * 128 + i0 + i] != 0
                                : (qi >= lo && qi <= hi));
          float s = 0.f;
#pragma unroll
          for (int d = 0; d < D; ++d) s = fmaf(kv[d], qs[i][d], s);
          s *= p.scale;
          if (p.cap > 0.f) s = p.cap * tanhf(s / p.cap);
          if (seen) w += expf(s - lse);
        }
      }
    }
  }
  p.out[(static_cast<int64_t>(b) * p.Hkv + g) * p.Skv + key] = w;
}

}  // namespace

size_t key_weights_workspace_bytes(const bsa_key_weights_args*, const bsa_mask_info*) { return 0; }

bsa_status key_weights_launch(const bsa_key_weights_args* a, const bsa_mask_info* info, float scale, cudaStream_t stream) {
  KeyWeightsParams p{};
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.k = static_cast<const __nv_bfloat16*>(a->k);
  p.lse = a->lse;
  p.q_lens = a->q_lens;
  p.out = a->weights;
  p.B = a->B;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.Sq = a->S_q;
  p.Skv = a->S_kv;
  p.scale = scale;
  p.cap = a->logits_soft_cap;
  p.mi = mask_info_dev(info);
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  const dim3 grid(static_cast<unsigned>(a->S_kv / 128), a->Hkv, a->B);
  cudaError_t e = a->D == 128 ? launch_kernel(key_weights_kernel<128>, grid, dim3(128), 0, stream, p)
                              : launch_kernel(key_weights_kernel<64>, grid, dim3(128), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "key weights launch");
  return BSA_OK;
}

}  // namespace bsa
