// Tables and slots of the cache in pages, from the sequences' lengths.
//
// With have = ceil(lens / page) and want = ceil(new_lens / page), sequence b gives back drop = max(have - want, 0) pages
// and needs need = max(want - have, 0).  After the pages given back, in order of (sequence, place), stand on the stack
// from `base` = used - sum(drop) on, the pages of sequence b are entries base + (sum of need before b) .., if the
// sum up to b fits, else it and every later one that needs pages waits.
//
// Every CTA forms the two prefix sums for itself (two arrays of B words, read from the second-level cache) and then
// places its share of the pages and slots.  A page that is given back and taken in the same call is looked up
// in the row that gives it (a binary search over the prefix sums), not on the stack, so no CTA waits for another: reads
// are of stack entries from `used` on and of table entries that are not written.
// 256 sequences that grow by a token take 3.9 us, 64 that take prompts of up to 8192 6.3 (2.2 MB): latency, of lengths, sums,
// table and slots one after the other.
#include <algorithm>

#include "paged.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxB = 4096;
constexpr int kChunk = 256;  // table entries, or slots, of one row that a warp takes at a time

struct ResizeParams {
  int32_t *table, *free_pages;
  const int32_t *used, *lens, *new_lens;
  int32_t *lens_out, *used_out, *slots;
  int32_t B, shift, pages;
  int64_t M, T;
  uint32_t* err;
};

// Sums stop at kMost, more than any stack holds (of absurd lengths they would not fit in 32 bits).
constexpr int32_t kMost = 1 << 30;
__device__ __forceinline__ int32_t sum(int32_t a, int32_t b) { return min(a + b, kMost); }

struct Row {
  int32_t len, next;    // tokens now, and to be
  int32_t have, want;   // pages
};

struct Tables {
  int32_t drop[kMaxB + 1];  // pages given back by the sequences before b
  int32_t need[kMaxB + 1];  // pages needed by the sequences before b
  int32_t sums[kThreads / 32][2];
};

__device__ __forceinline__ Row load_row(const ResizeParams& p, int32_t b, uint32_t* err) {
  Row r;
  r.len = p.lens[b];
  r.next = p.new_lens[b];
  const int64_t most = p.M << p.shift;
  const bool fits = r.len >= 0 && r.len <= most && r.next >= 0 && r.next <= most && static_cast<int64_t>(r.next) - r.len <= p.T;
  if (!fits) {
    if (err) atomicOr(err, DEV_ERR_BOUNDS);
    r.next = r.len;
    r.have = r.want = 0;
    return r;
  }
  const int32_t up = (1 << p.shift) - 1;
  r.have = static_cast<int32_t>((static_cast<int64_t>(r.len) + up) >> p.shift);
  r.want = static_cast<int32_t>((static_cast<int64_t>(r.next) + up) >> p.shift);
  return r;
}

__device__ __forceinline__ int32_t checked_page(const ResizeParams& p, int32_t page) {
  if ((page < 0 || page >= p.pages) && p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
  return page;
}

// Entry i of the stack once the pages given back are on it.
__device__ __forceinline__ int32_t on_stack(const ResizeParams& p, const Tables& t, int32_t base, int32_t used, int32_t i) {
  if (i >= used) return p.free_pages[i];
  int32_t lo = 0, hi = p.B;  // the last sequence whose pages begin at or before i - base
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) / 2;
    if (t.drop[mid] <= i - base) lo = mid;
    else hi = mid;
  }
  return p.table[lo * p.M + load_row(p, lo, nullptr).want + (i - base - t.drop[lo])];
}

__global__ void __launch_bounds__(kThreads) resize_kernel(const __grid_constant__ ResizeParams p) {
  __shared__ Tables t;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool first_cta = blockIdx.x == 0;
  // ---- prefix sums: a run of sequences a thread
  const int32_t per = (p.B + kThreads - 1) / kThreads, b0 = static_cast<int32_t>(threadIdx.x) * per, b1 = min(b0 + per, p.B);
  int32_t drop = 0, need = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const Row r = load_row(p, b, first_cta ? p.err : nullptr);
    drop = sum(drop, max(r.have - r.want, 0));
    need = sum(need, max(r.want - r.have, 0));
  }
  int32_t id = drop, in = need;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int32_t xd = __shfl_up_sync(0xffffffffu, id, o), xn = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) {
      id = sum(id, xd);
      in = sum(in, xn);
    }
  }
  if (lane == 31) {
    t.sums[warp][0] = id;
    t.sums[warp][1] = in;
  }
  __syncthreads();
  int32_t all_drop = 0, all_need = 0;
  drop = __shfl_up_sync(0xffffffffu, id, 1);
  need = __shfl_up_sync(0xffffffffu, in, 1);
  if (lane == 0) drop = need = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) {
      drop = sum(drop, all_drop);
      need = sum(need, all_need);
    }
    all_drop = sum(all_drop, t.sums[w][0]);
    all_need = sum(all_need, t.sums[w][1]);
  }
  for (int32_t b = b0; b < b1; ++b) {
    const Row r = load_row(p, b, nullptr);
    t.drop[b] = drop;
    t.need[b] = need;
    drop = sum(drop, max(r.have - r.want, 0));
    need = sum(need, max(r.want - r.have, 0));
  }
  if (threadIdx.x == 0) {
    t.drop[p.B] = all_drop;
    t.need[p.B] = all_need;
  }
  __syncthreads();
  const int32_t used = p.used[0];
  const bool usable = used >= 0 && used <= p.pages && all_drop <= used;
  const int32_t base = used - all_drop, room = p.pages - base;
  if (!usable) {
    if (first_cta && threadIdx.x == 0) {
      if (p.err) atomicOr(p.err, DEV_ERR_BOUNDS);
      p.used_out[0] = used;
    }
  } else if (first_cta && threadIdx.x == 0) {
    // the sums of those that fit: the largest prefix sum that does
    int32_t lo = 0, hi = p.B;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) / 2;
      if (t.need[mid] <= room) lo = mid;
      else hi = mid - 1;
    }
    p.used_out[0] = base + t.need[lo];
  }
  // ---- a warp takes a piece of a row: kChunk entries of the table and kChunk slots
  const int64_t pieces = (max(p.M, p.T) + kChunk - 1) / kChunk;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp; u < pieces * p.B; u += step) {
    const int32_t b = static_cast<int32_t>(u / pieces);
    const int64_t c0 = (u - b * pieces) * kChunk;
    Row r = load_row(p, b, nullptr);
    if (!usable || (r.want > r.have && t.need[b + 1] > room)) {
      r.next = r.len;
      r.want = r.have;
    }
    if (c0 == 0 && lane == 0) p.lens_out[b] = r.next;
    int32_t* row = p.table + b * p.M;
    const int32_t m1 = static_cast<int32_t>(min(c0 + kChunk, p.M));
    // (sums are of what was asked for: equal to what is done, for every sequence that is served)
    for (int32_t j = max(static_cast<int32_t>(c0), r.want) + lane; j < min(m1, r.have); j += 32)
      p.free_pages[base + t.drop[b] + (j - r.want)] = checked_page(p, row[j]);
    for (int32_t j = max(static_cast<int32_t>(c0), r.have) + lane; j < min(m1, r.want); j += 32)
      row[j] = checked_page(p, on_stack(p, t, base, used, base + t.need[b] + (j - r.have)));
    const int64_t fresh = max(r.next - r.len, 0);
    for (int64_t i = c0 + lane; i < min(c0 + kChunk, p.T); i += 32) {
      int32_t slot = -1;
      if (i < fresh) {
        const int32_t at = r.len + static_cast<int32_t>(i), j = at >> p.shift;
        const int32_t page = checked_page(p, j < r.have ? row[j] : on_stack(p, t, base, used, base + t.need[b] + (j - r.have)));
        if (page >= 0 && page < p.pages) slot = (page << p.shift) + (at & ((1 << p.shift) - 1));
      }
      p.slots[b * p.T + i] = slot;
    }
  }
}

}  // namespace

bsa_status paged_resize_launch(const bsa_paged_resize_args* a, cudaStream_t stream) {
  ResizeParams p{};
  p.table = a->table;
  p.free_pages = a->free_pages;
  p.used = a->used;
  p.lens = a->lens;
  p.new_lens = a->new_lens;
  p.lens_out = a->lens_out;
  p.used_out = a->used_out;
  p.slots = a->slots;
  p.B = a->B;
  p.shift = page_shift(a->page);
  p.pages = static_cast<int32_t>(a->pages);
  p.M = a->M;
  p.T = a->T;
  p.err = device_error_word();
  if (!p.err) return fail(BSA_ERR_CUDA, "could not allocate the device error word");
  const int64_t pieces = a->B * ((std::max(a->M, a->T) + kChunk - 1) / kChunk), per = kThreads / 32;
  const int grid = static_cast<int>(std::min<int64_t>((pieces + per - 1) / per, static_cast<int64_t>(num_sms()) * 4));
  cudaError_t e = launch_kernel(resize_kernel, dim3(grid), dim3(kThreads), 0, stream, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged resize launch");
  return BSA_OK;
}

}  // namespace bsa
