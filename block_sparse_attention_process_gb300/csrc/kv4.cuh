// The 4-bit key/value cache: row layout and quantisation shared by the
// append, attention and eviction kernels.
//
// A row of D elements is D/32 groups of 32, each with one bf16 scale s and 4-bit
// codes c (value s * (c - 8)).  The order of the codes within a row makes the
// fragments of m16n8k16 products plain loads:
//  * K row, 4-byte word t * (D/32) + g (t = 0..3): elements 32 g + 8 t + 0..7.
//    Thread t of a fragment row finds its eight elements of every group in
//    D/8 consecutive bytes.
//  * V row, 2-byte word p * (D/32) + g (p = 0..7): elements 32 g + 4 p + 0..3,
//    so the eight fragment rows p find their four elements of every group in
//    D/16 consecutive bytes.  With D = 128 the row's two 32-byte halves are
//    exchanged in slots with bit 1 set: the four keys whose rows are read
//    together (one per value of t) then lie in different shared-memory banks.
#pragma once
#include <cstdint>

#include "bsa.h"
#include "internal.h"
#include "ptx.cuh"

namespace bsa {

constexpr int kKv4Group = 32;

template <int D>
struct Kv4 {
  static constexpr int kGroups = D / 32;
  static constexpr int kRowBytes = D / 2;       // codes of one key or value
  static constexpr int kScaleBytes = D / 16;    // scales of one key or value
  static constexpr int kWords = D / 8;          // 32-bit words of codes in a row
  static constexpr int kPieceWords = D / 64;    // 32-bit words per V piece p
};

// Exchange of a V row's halves, as an XOR of its 32-bit word index.
template <int D>
__device__ __forceinline__ uint32_t v_word_swap(int64_t slot) {
  return D == 128 ? static_cast<uint32_t>(slot & 2) << 2 : 0u;
}

// First element of 32-bit word w of a K row (8 elements follow), and of the
// two groups of four in word w of an (unswapped) V row.
template <int D>
__device__ __forceinline__ int k_word_elem(int w) {
  return 32 * (w % Kv4<D>::kGroups) + 8 * (w / Kv4<D>::kGroups);
}
template <int D>
__device__ __forceinline__ int v_word_elem(int w, int half) {
  return 32 * (2 * (w % Kv4<D>::kPieceWords) + half) + 4 * (w / Kv4<D>::kPieceWords);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A device-side length or slot count brought into [0, hi]; one outside sets
// the bounds bit.
__device__ __forceinline__ int32_t clamp_len(int32_t n, int64_t hi, uint32_t* err) {
  if (n < 0 || n > hi) {
    if (err) atomicOr(err, DEV_ERR_BOUNDS);
    return n < 0 ? 0 : static_cast<int32_t>(hi);
  }
  return n;
}

}  // namespace bsa
