// The cache in pages: what its kernels share.
#pragma once
#include <cstdint>

#include "bsa.h"
#include "internal.h"
#include "ptx.cuh"

namespace bsa {

// A device-side length brought into [0, hi]; one outside sets the bounds bit.
__device__ __forceinline__ int32_t paged_len(int32_t n, int64_t hi, uint32_t* err) {
  if (n < 0 || n > hi) {
    if (err) atomicOr(err, DEV_ERR_BOUNDS);
    return n < 0 ? 0 : static_cast<int32_t>(hi);
  }
  return n;
}

// 2^max(floor(log2 top) - bits, -100) and its inverse, of 0 <= top < 2^100; both are normal numbers.
__device__ __forceinline__ void unit_of(float top, int bits, float& unit, float& inverse) {
  const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - bits, -100);
  unit = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  inverse = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}
constexpr float kUsualTop = 0x1p100f;  // keys (or queries) below this have bounds (or codes)

// Division of 0 <= n < 2^31 by a number known on the host, as a product: with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// n / d = (n m / 2^32 + n) / 2^l, rounded down both times.
struct Divisor {
  uint32_t m = 1, l = 0;
  Divisor() = default;
  explicit Divisor(uint32_t d) {
    while (l < 31 && (uint32_t(1) << l) < d) ++l;
    m = static_cast<uint32_t>((((uint64_t(1) << l) - d) << 32) / d) + 1;
  }
  __device__ __forceinline__ int32_t of(int32_t n) const {
    return static_cast<int32_t>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> l);
  }
};

// log2 of a page size (16 .. 256)
inline int page_shift(int32_t page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

}  // namespace bsa
