// C entry points of the calls that follow a prompt: key weights and the
// 4-bit cache (append, attention, eviction).  Argument checks and dispatch.
#include <cmath>

#include "internal.h"

namespace bsa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bsa_status bad(const char* msg) { return fail(BSA_ERR_INVALID_ARG, msg); }

// No exception leaves a C entry (message strings may fail to allocate).
template <typename F>
bsa_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return BSA_ERR_OOM;
  }
}

bsa_status check_cache(const bsa_kv4_cache& c) {
  if (c.B <= 0 || c.Hkv <= 0) return bad("B and Hkv must be positive");
  if (c.D != 64 && c.D != 128) return fail(BSA_ERR_UNSUPPORTED, "head dim must be 64 or 128");
  if (c.capacity <= 0 || c.capacity % 16) return bad("capacity must be a positive multiple of 16");
  if (c.capacity > (int64_t(1) << 30)) return fail(BSA_ERR_UNSUPPORTED, "capacity above 2^30 is not supported");
  if (static_cast<int64_t>(c.B) * c.Hkv > INT32_MAX) return fail(BSA_ERR_UNSUPPORTED, "B*Hkv must fit in int32");
  const void* ptrs[] = {c.k_codes, c.k_scales, c.v_codes, c.v_scales};
  for (const void* p : ptrs) {
    if (!p) return bad("a cache pointer is null");
    if (!aligned16(p)) return bad("cache codes and scales must be 16-byte aligned");
  }
  if (!aligned4(c.weights) || !aligned4(c.positions)) return bad("cache weights and positions must be 4-byte aligned");
  return BSA_OK;
}

bsa_status check_strides(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] % 8) return bad("strides must be multiples of 8 elements");
  return BSA_OK;
}

bsa_status check_cap(float cap) {
  if (!(cap >= 0.f) || std::isinf(cap)) return bad("logits_soft_cap must be finite and >= 0");
  return BSA_OK;
}

float resolve_scale(float s, int32_t D) { return std::isnan(s) ? 1.0f / std::sqrt(static_cast<float>(D)) : s; }

bsa_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return BSA_OK;
  if (!ws || have < need) return bad("the workspace is missing or smaller than the call needs");
  if (!aligned16(ws)) return bad("the workspace must be 16-byte aligned");
  return BSA_OK;
}

bsa_status check_append(const bsa_kv4_append_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_cache(a->cache);
  if (s != BSA_OK) return s;
  if (a->T <= 0) return bad("T must be positive");
  if (static_cast<int64_t>(a->cache.B) * a->cache.Hkv > INT32_MAX / a->T)
    return fail(BSA_ERR_UNSUPPORTED, "B*Hkv*T must fit in int32");
  if (!a->k || !a->v || !a->start) return bad("k, v and start must be non-null");
  if (!aligned16(a->k) || !aligned16(a->v) || !aligned16(a->k_values) || !aligned16(a->v_values))
    return bad("k, v and their values must be 16-byte aligned");
  if (!aligned4(a->start) || !aligned4(a->n_new) || !aligned4(a->first_position) || !aligned4(a->weights0))
    return bad("start, n_new, first_position and weights0 must be 4-byte aligned");
  s = check_strides(a->k_stride);
  return s != BSA_OK ? s : check_strides(a->v_stride);
}

bsa_status check_fwd(const bsa_kv4_fwd_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_cache(a->cache);
  if (s != BSA_OK) return s;
  if (a->Hq <= 0 || a->Hq % a->cache.Hkv) return bad("Hq must be a positive multiple of Hkv");
  if (a->T <= 0) return bad("T must be positive");
  if (static_cast<int64_t>(a->cache.B) * a->Hq > INT32_MAX / a->T)
    return fail(BSA_ERR_UNSUPPORTED, "B*Hq*T must fit in int32");
  if (!kv4_fwd_fits(a)) return fail(BSA_ERR_UNSUPPORTED, "too many rows or slots for one launch");
  if (a->accumulate != 0 && a->accumulate != 1) return bad("accumulate must be 0 or 1");
  if (a->accumulate && !a->cache.weights) return bad("accumulate needs the cache's weights");
  s = check_cap(a->logits_soft_cap);
  if (s != BSA_OK) return s;
  if (a->num_sinks < 0 || a->num_sinks > 64) return fail(BSA_ERR_UNSUPPORTED, "num_sinks must be in 0..64");
  if (a->num_sinks > 0 && !a->sinks) return bad("sinks is null");
  if (!aligned4(a->sinks)) return bad("sinks must be 4-byte aligned");
  return BSA_OK;
}

bsa_status check_fwd_tensors(const bsa_kv4_fwd_args* a) {
  if (!a->q || !a->o || !a->lse || !a->lens) return bad("q, o, lse and lens must be non-null");
  if (!aligned16(a->q) || !aligned16(a->o)) return bad("q and o must be 16-byte aligned");
  if (!aligned4(a->lse) || !aligned4(a->lens) || !aligned4(a->q_lens)) return bad("lse, lens and q_lens must be 4-byte aligned");
  bsa_status s = check_strides(a->q_stride);
  if (s == BSA_OK) s = check_strides(a->o_stride);
  if (s != BSA_OK) return s;
  const int64_t rows[] = {a->cache.B, a->Hq, a->T};
  for (int i = 0; i < 3; ++i)
    if (rows[i] > 1 && a->o_stride[i] == 0) return bad("o must not have several rows in one place");
  return BSA_OK;
}

bsa_status check_evict(const bsa_kv4_evict_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_cache(a->cache);
  if (s != BSA_OK) return s;
  s = check_cache(a->out);
  if (s != BSA_OK) return s;
  const bsa_kv4_cache &c = a->cache, &o = a->out;
  if (c.B != o.B || c.Hkv != o.Hkv || c.D != o.D) return bad("out must have the cache's B, Hkv and D");
  if (!c.weights) return bad("eviction needs the cache's weights");
  if (a->keep < 1) return bad("keep must be at least 1");
  if (a->keep > o.capacity) return bad("keep exceeds the capacity of out");
  if (a->recent < 0 || a->recent > a->keep) return bad("recent must be in 0..keep");
  const bool same[] = {c.k_codes == o.k_codes, c.k_scales == o.k_scales, c.v_codes == o.v_codes, c.v_scales == o.v_scales};
  const int n_same = same[0] + same[1] + same[2] + same[3];
  if (n_same != 0 && n_same != 4) return bad("out shares some of the cache's buffers: all or none");
  const bool in_place = n_same == 4;
  if (in_place && (c.capacity != o.capacity || c.weights != o.weights || c.positions != o.positions))
    return bad("in place, out must be the cache itself");
  if (!in_place && (c.weights == o.weights || (c.positions && c.positions == o.positions)))
    return bad("out shares some of the cache's buffers: all or none");
  if (in_place && a->recent > 0 && !c.positions) return bad("evicting in place with recent > 0 needs positions");
  if (static_cast<int64_t>(c.B) * c.Hkv > INT32_MAX / a->keep) return fail(BSA_ERR_UNSUPPORTED, "B*Hkv*keep must fit in int32");
  return BSA_OK;
}

bsa_status check_key_weights(const bsa_key_weights_args* a, const bsa_mask_info* info) {
  if (!a) return bad("args is null");
  if (a->B <= 0 || a->Hq <= 0 || a->Hkv <= 0) return bad("B, Hq and Hkv must be positive");
  if (a->Hq % a->Hkv) return bad("Hq must be a multiple of Hkv");
  if (a->S_q <= 0 || a->S_kv <= 0 || a->S_q % kBlock || a->S_kv % kBlock)
    return bad("sequence lengths must be positive multiples of 128");
  if (a->D != 64 && a->D != 128) return fail(BSA_ERR_UNSUPPORTED, "head dim must be 64 or 128");
  if (static_cast<int64_t>(a->B) * a->Hq > INT32_MAX / a->S_q || static_cast<int64_t>(a->B) * a->Hkv > INT32_MAX / a->S_kv)
    return fail(BSA_ERR_UNSUPPORTED, "B*H*S must fit in int32");
  bsa_status s = check_cap(a->logits_soft_cap);
  if (s != BSA_OK) return s;
  if (a->S_q / kBlock > 65536) return fail(BSA_ERR_UNSUPPORTED, "more than 65536 query blocks are not supported");  // (16 bits of an item)
  if (!info) return bad("dkv MaskInfo is null");
  return BSA_OK;
}

bsa_status check_key_weights_info(const bsa_key_weights_args* a, const bsa_mask_info* info) {
  if (info->orientation != BSA_ORIENT_DKV) return bad("dkv MaskInfo has the wrong orientation");
  if (info->q_len != a->S_q || info->kv_len != a->S_kv) return bad("dkv MaskInfo was compiled for other sequence lengths");
  if (info->heads != 1 && info->heads != a->Hq) return bad("dkv MaskInfo must have 1 or Hq mask heads");
  return BSA_OK;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsa_kv4_append(const bsa_kv4_append_args* a, bsa_stream stream) {
  return guarded([&] {
    const bsa_status s = check_append(a);
    return s != BSA_OK ? s : kv4_append_launch(a, static_cast<cudaStream_t>(stream));
  });
}

bsa_status bsa_kv4_fwd_workspace(const bsa_kv4_fwd_args* a, size_t* bytes) {
  return guarded([&] {
    if (!bytes) return bad("bytes is null");
    const bsa_status s = check_fwd(a);
    if (s == BSA_OK) *bytes = kv4_fwd_workspace_bytes(a);
    return s;
  });
}

bsa_status bsa_kv4_fwd(const bsa_kv4_fwd_args* a, bsa_stream stream) {
  return guarded([&] {
    bsa_status s = check_fwd(a);
    if (s == BSA_OK) s = check_fwd_tensors(a);
    if (s == BSA_OK) s = check_workspace(a->workspace, a->workspace_bytes, kv4_fwd_workspace_bytes(a));
    return s != BSA_OK ? s : kv4_fwd_launch(a, resolve_scale(a->softmax_scale, a->cache.D), static_cast<cudaStream_t>(stream));
  });
}

bsa_status bsa_kv4_evict_workspace(const bsa_kv4_evict_args* a, size_t* bytes) {
  return guarded([&] {
    if (!bytes) return bad("bytes is null");
    const bsa_status s = check_evict(a);
    if (s == BSA_OK) *bytes = kv4_evict_workspace_bytes(a);
    return s;
  });
}

bsa_status bsa_kv4_evict(const bsa_kv4_evict_args* a, bsa_stream stream) {
  return guarded([&] {
    bsa_status s = check_evict(a);
    if (s != BSA_OK) return s;
    if (!a->lens || !a->new_lens || !a->index) return bad("lens, new_lens and index must be non-null");
    // (other heads' CTAs still read the lengths)
    if (a->new_lens == a->lens || a->new_lens == a->seen) return bad("new_lens must be neither lens nor seen");
    if (!aligned4(a->lens) || !aligned4(a->seen) || !aligned4(a->new_lens) || !aligned4(a->index))
      return bad("lens, seen, new_lens and index must be 4-byte aligned");
    if (!aligned16(a->k_values) || !aligned16(a->v_values)) return bad("values must be 16-byte aligned");
    s = check_workspace(a->workspace, a->workspace_bytes, kv4_evict_workspace_bytes(a));
    return s != BSA_OK ? s : kv4_evict_launch(a, static_cast<cudaStream_t>(stream));
  });
}

bsa_status bsa_key_weights_workspace(const bsa_key_weights_args* a, const bsa_mask_info* info, size_t* bytes) {
  return guarded([&] {
    if (!bytes) return bad("bytes is null");
    bsa_status s = check_key_weights(a, info);
    if (s == BSA_OK) s = check_key_weights_info(a, info);
    if (s == BSA_OK) *bytes = key_weights_workspace_bytes(a, info);
    return s;
  });
}

bsa_status bsa_key_weights(const bsa_key_weights_args* a, const bsa_mask_info* info, bsa_stream stream) {
  return guarded([&] {
    bsa_status s = check_key_weights(a, info);
    if (s != BSA_OK) return s;
    if (!a->q || !a->k || !a->lse || !a->weights) return bad("a tensor pointer is null");
    if (!aligned16(a->q) || !aligned16(a->k) || !aligned16(a->lse) || !aligned16(a->weights))
      return bad("tensor pointers must be 16-byte aligned");
    if (!aligned4(a->q_lens)) return bad("q_lens must be 4-byte aligned");
    s = check_key_weights_info(a, info);
    if (s == BSA_OK) s = check_workspace(a->workspace, a->workspace_bytes, key_weights_workspace_bytes(a, info));
    return s != BSA_OK ? s : key_weights_launch(a, info, resolve_scale(a->softmax_scale, a->D), static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
