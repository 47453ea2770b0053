// C entry points of the cache in pages: tables, append, selection, attention.
// Argument checks and dispatch.
#include <cmath>

#include "internal.h"

namespace bsa {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bsa_status bad(const char* msg) { return fail(BSA_ERR_INVALID_ARG, msg); }
bsa_status unsupported(const char* msg) { return fail(BSA_ERR_UNSUPPORTED, msg); }

// No exception leaves a C entry (message strings may fail to allocate).
template <typename F>
bsa_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return BSA_ERR_OOM;
  }
}

bsa_status check_pages(int64_t pages, int32_t page) {
  if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256)
    return unsupported("a page must hold 16, 32, 64, 128 or 256 tokens");
  if (pages <= 0) return bad("pages must be positive");
  if (pages > INT32_MAX / page) return unsupported("pages times tokens of a page must fit in int32");
  return BSA_OK;
}

bsa_status check_cache(const bsa_paged_cache& c, bool need_kv) {
  const bsa_status s = check_pages(c.pages, c.page);
  if (s != BSA_OK) return s;
  if (c.Hkv <= 0) return bad("Hkv must be positive");
  if (c.D != 64 && c.D != 128) return unsupported("head dim must be 64 or 128");
  if (!aligned16(c.bounds)) return bad("bounds must be 16-byte aligned");
  if (!need_kv) return BSA_OK;
  if (!c.k || !c.v) return bad("a cache pointer is null");
  if (!aligned16(c.k) || !aligned16(c.v)) return bad("the cache's k and v must be 16-byte aligned");
  const int64_t n[] = {c.pages, c.Hkv, c.page};
  for (const int64_t* st : {c.k_stride, c.v_stride})
    for (int i = 0; i < 3; ++i) {
      if (st[i] < 0 || st[i] % 8) return bad("the cache's strides must be non-negative multiples of 8 elements");
      if (st[i] >= (int64_t(1) << 35)) return unsupported("the cache's strides must be below 2^35 elements");  // (in 16 bytes: 32 bits)
      if (n[i] > 1 && st[i] == 0) return bad("the cache must not have several rows in one place");
    }
  return BSA_OK;
}

bsa_status check_strides(const int64_t* s) {
  for (int i = 0; i < 3; ++i)
    if (s[i] % 8) return bad("strides must be multiples of 8 elements");
  return BSA_OK;
}

bsa_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return BSA_OK;
  if (!ws || have < need) return bad("the workspace is missing or smaller than the call needs");
  if (!aligned16(ws)) return bad("the workspace must be 16-byte aligned");
  return BSA_OK;
}

constexpr int64_t kMostTokens = int64_t(1) << 30;  // of a sequence

bsa_status check_table(int64_t M, int32_t page) {
  if (M <= 0) return bad("M must be positive");
  if (M > kMostTokens / page) return unsupported("M pages must hold at most 2^30 tokens");
  return BSA_OK;
}

bsa_status check_queries(int32_t B, int32_t Hq, int32_t Hkv, int64_t T) {
  if (B <= 0) return bad("B must be positive");
  if (Hq <= 0 || Hq % Hkv) return bad("Hq must be a positive multiple of Hkv");
  if (T <= 0) return bad("T must be positive");
  if (static_cast<int64_t>(B) * Hq > INT32_MAX / T) return unsupported("B*Hq*T must fit in int32");
  return BSA_OK;
}

bsa_status check_resize(const bsa_paged_resize_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_pages(a->pages, a->page);
  if (s == BSA_OK) s = check_table(a->M, a->page);
  if (s != BSA_OK) return s;
  if (a->B <= 0) return bad("B must be positive");
  if (a->B > 4096) return unsupported("more than 4096 sequences are not supported");
  if (a->T <= 0) return bad("T must be positive");
  if (a->T > INT32_MAX / a->B) return unsupported("B*T must fit in int32");
  const void* in[] = {a->table, a->free_pages, a->used, a->lens, a->new_lens};
  const void* out[] = {a->lens_out, a->used_out, a->slots};
  for (const void* p : in)
    if (!p || !aligned4(p)) return bad("table, free_pages, used, lens and new_lens must be non-null and 4-byte aligned");
  for (int i = 0; i < 3; ++i) {
    if (!out[i] || !aligned4(out[i])) return bad("lens_out, used_out and slots must be non-null and 4-byte aligned");
    // (other CTAs still read the inputs)
    for (const void* p : in)
      if (p == out[i]) return bad("an output of the resize must not be the memory of an input");
    for (int j = 0; j < i; ++j)
      if (out[i] == out[j]) return bad("two outputs of the resize are the same memory");
  }
  if (a->table == a->free_pages) return bad("table and free_pages are the same memory");
  return BSA_OK;
}

bsa_status check_append(const bsa_paged_append_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_cache(a->cache, true);
  if (s != BSA_OK) return s;
  s = check_queries(a->B, a->cache.Hkv, a->cache.Hkv, a->T);
  if (s != BSA_OK) return s;
  if (a->cache.bounds && paged_append_units(a) > INT32_MAX / (static_cast<int64_t>(a->B) * a->cache.Hkv))
    return unsupported("too many pages for one launch");
  if (!a->k || !a->v || !a->slots) return bad("k, v and slots must be non-null");
  if (!aligned16(a->k) || !aligned16(a->v)) return bad("k and v must be 16-byte aligned");
  if (!aligned4(a->slots)) return bad("slots must be 4-byte aligned");
  s = check_strides(a->src_k_stride);
  return s != BSA_OK ? s : check_strides(a->src_v_stride);
}

bsa_status check_select(const bsa_paged_select_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_cache(a->cache, false);
  if (s != BSA_OK) return s;
  if (!a->cache.bounds) return bad("selection needs the cache's bounds");
  s = check_queries(a->B, a->Hq, a->cache.Hkv, a->T);
  if (s == BSA_OK) s = check_table(a->M, a->cache.page);
  if (s != BSA_OK) return s;
  if (a->first < 0 || a->recent < 0) return bad("first and recent must not be negative");
  if (a->keep < 1) return bad("keep must be at least 1");
  if (a->first > a->keep || a->recent > a->keep - a->first) return bad("keep must be at least first + recent");
  if (a->keep > INT32_MAX / (static_cast<int64_t>(a->B) * a->cache.Hkv * a->T)) return unsupported("B*Hkv*T*keep must fit in int32");
  if (!paged_select_fits(a)) return unsupported("more than 49152 pages a sequence, or too many queries for one launch");
  return BSA_OK;
}

bsa_status check_fwd(const bsa_paged_fwd_args* a) {
  if (!a) return bad("args is null");
  bsa_status s = check_cache(a->cache, true);
  if (s != BSA_OK) return s;
  s = check_queries(a->B, a->Hq, a->cache.Hkv, a->T);
  if (s == BSA_OK) s = check_table(a->M, a->cache.page);
  if (s != BSA_OK) return s;
  if (a->kind != BSA_MASK_CAUSAL && a->kind != BSA_MASK_LOCAL && a->kind != BSA_MASK_CHUNKED_CAUSAL)
    return unsupported("kind must be causal, local or chunked causal");
  if (a->kind == BSA_MASK_LOCAL && a->local_left < -1) return bad("local_left must be -1 or not negative");
  if (a->kind == BSA_MASK_CHUNKED_CAUSAL && a->chunk <= 0) return bad("chunk must be positive");
  if (a->select) {
    if (a->kind != BSA_MASK_CAUSAL) return unsupported("lists of pages go with the causal kind");
    if (a->keep < 1) return bad("keep must be at least 1");
    if (a->keep > kMostTokens / a->cache.page) return unsupported("keep pages must hold at most 2^30 tokens");
    if (!aligned4(a->select)) return bad("select must be 4-byte aligned");
  }
  if (!paged_fwd_fits(a)) return unsupported("too many rows for one launch");
  if (!(a->logits_soft_cap >= 0.f) || std::isinf(4.0f * a->logits_soft_cap)) return bad("logits_soft_cap must be >= 0 and below 2^126");
  if (a->num_sinks < 0 || a->num_sinks > 64) return unsupported("num_sinks must be in 0..64");
  if (a->num_sinks > 0 && !a->sinks) return bad("sinks is null");
  if (!aligned4(a->sinks)) return bad("sinks must be 4-byte aligned");
  return BSA_OK;
}

bsa_status check_fwd_tensors(const bsa_paged_fwd_args* a) {
  if (!a->q || !a->o || !a->lse || !a->lens || !a->table) return bad("q, o, lse, lens and table must be non-null");
  if (!aligned16(a->q) || !aligned16(a->o)) return bad("q and o must be 16-byte aligned");
  if (!aligned4(a->lse) || !aligned4(a->lens) || !aligned4(a->q_lens) || !aligned4(a->table))
    return bad("lse, lens, q_lens and table must be 4-byte aligned");
  bsa_status s = check_strides(a->q_stride);
  if (s == BSA_OK) s = check_strides(a->o_stride);
  if (s != BSA_OK) return s;
  const int64_t rows[] = {a->B, a->Hq, a->T};
  for (int i = 0; i < 3; ++i)
    if (rows[i] > 1 && a->o_stride[i] == 0) return bad("o must not have several rows in one place");
  return BSA_OK;
}

}  // namespace
}  // namespace bsa

using namespace bsa;

extern "C" {

bsa_status bsa_paged_resize(const bsa_paged_resize_args* a, bsa_stream stream) {
  return guarded([&] {
    const bsa_status s = check_resize(a);
    return s != BSA_OK ? s : paged_resize_launch(a, static_cast<cudaStream_t>(stream));
  });
}

bsa_status bsa_paged_append(const bsa_paged_append_args* a, bsa_stream stream) {
  return guarded([&] {
    const bsa_status s = check_append(a);
    return s != BSA_OK ? s : paged_append_launch(a, static_cast<cudaStream_t>(stream));
  });
}

bsa_status bsa_paged_select(const bsa_paged_select_args* a, bsa_stream stream) {
  return guarded([&] {
    bsa_status s = check_select(a);
    if (s != BSA_OK) return s;
    if (!a->q || !a->table || !a->lens || !a->index) return bad("q, table, lens and index must be non-null");
    if (!aligned16(a->q)) return bad("q must be 16-byte aligned");
    if (!aligned4(a->table) || !aligned4(a->lens) || !aligned4(a->q_lens) || !aligned4(a->index))
      return bad("table, lens, q_lens and index must be 4-byte aligned");
    s = check_strides(a->q_stride);
    return s != BSA_OK ? s : paged_select_launch(a, static_cast<cudaStream_t>(stream));
  });
}

bsa_status bsa_paged_fwd_workspace(const bsa_paged_fwd_args* a, size_t* bytes) {
  return guarded([&] {
    if (!bytes) return bad("bytes is null");
    const bsa_status s = check_fwd(a);
    if (s == BSA_OK) *bytes = paged_fwd_workspace_bytes(a);
    return s;
  });
}

bsa_status bsa_paged_fwd(const bsa_paged_fwd_args* a, bsa_stream stream) {
  return guarded([&] {
    bsa_status s = check_fwd(a);
    if (s == BSA_OK) s = check_fwd_tensors(a);
    if (s == BSA_OK) s = check_workspace(a->workspace, a->workspace_bytes, paged_fwd_workspace_bytes(a));
    if (s != BSA_OK) return s;
    const float scale = std::isnan(a->softmax_scale) ? 1.0f / std::sqrt(static_cast<float>(a->cache.D)) : a->softmax_scale;
    if (!std::isfinite(4.0f * scale) || (a->logits_soft_cap > 0.f && !std::isfinite(4.0f * (scale / a->logits_soft_cap))))
      return bad("softmax_scale, and softmax_scale over the cap, must be finite");  // (times 2 log2 e)
    return paged_fwd_launch(a, scale, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
