// Division by numbers that a launch fixes.
#pragma once

#include <cstdint>

namespace qsfm {

// Division of 31-bit numbers by an invariant d: q = (n * m) >> (32 + s) with
// m = ceil(2^(32 + s) / d), s = ceil(log2 d) - 1 (exact for n < 2^31).
struct FastDiv {
  uint32_t d, m, s;
  __host__ void set(uint32_t div) {
    d = div;
    s = 0;
    while ((2u << s) < div) ++s;
    m = div <= 1 ? 0 : uint32_t(((1ull << (32 + s)) + div - 1) / div);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d <= 1 ? n : __umulhi(n, m) >> s; }
};

}  // namespace qsfm
