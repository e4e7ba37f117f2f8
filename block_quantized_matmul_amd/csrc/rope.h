// Rotation angles as fractions of a turn (host side).
#pragma once

#include <stdint.h>

namespace qmm {

// f / 2 pi in units of 2^-64, modulo 1, to within a unit: f is m 2^e with a
// 53-bit integer m, and m 2^65 / pi an integer product of 117 bits.
inline uint64_t to_turn(double f) {
  const uint64_t bits = __builtin_bit_cast(uint64_t, f);
  const int e = static_cast<int>(bits >> 52 & 0x7FF);
  if (e == 0) return 0;  // zero, or far below any angle
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull;
  const unsigned __int128 product = static_cast<unsigned __int128>(m) * 0xA2F9836E4E44152Aull;  // 2^65 / pi
  const int shift = 1077 - e;  // f = m 2^(e - 1075); 64 fraction bits, and 66 in the constant
  uint64_t t = 0;
  if (shift < 128)  // and above 47, |f| being at most 64
    t = static_cast<uint64_t>((product + (static_cast<unsigned __int128>(1) << (shift - 1))) >> shift);
  return f < 0 ? 0 - t : t;
}

}  // namespace qmm
