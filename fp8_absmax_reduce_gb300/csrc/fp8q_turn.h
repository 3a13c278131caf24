// Rotary frequencies as fixed-point fractions of a turn (host arithmetic, no CUDA).
#pragma once

#include <cmath>
#include <cstdint>

namespace fp8q {

// freq (radians per position, finite) in turns per position modulo one turn, in units of 2^-64, rounded to the nearest.
// The fraction is taken of |freq| / 2 pi, where it is exact, and a negative frequency negates the integer: the fraction
// of a small negative number itself lies next to 1, where doubles are 2^-53 apart, or is 1.
inline uint64_t rope_turn(double freq) {
  const double turns = std::fabs(freq) / 6.283185307179586476925;
  // at most 1 - 2^-53, so the product is below 2^64, and a whole number from 2^53 on
  const uint64_t u = (uint64_t)std::round((turns - std::floor(turns)) * 18446744073709551616.0);
  return freq < 0.0 ? (uint64_t)0 - u : u;
}

}  // namespace fp8q
