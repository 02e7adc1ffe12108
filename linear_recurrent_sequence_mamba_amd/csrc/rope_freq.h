// rope_freq.h -- turns per position of the rotary pairs.  Not part of the
// public ABI.
#pragma once

#include <math.h>

namespace m3 {

// f[j] = base^(-2 j / rot) / (2 pi) for j < rot / 2 <= 128.  A position up to 2^31
// multiplies the error, so it must not grow from pair to pair: each is the product
// of two powers, of a multiple of eight and of the rest, within 7 + (2 j / rot)
// |ln base| half steps of fp64 (at 2^31 - 1 and base 1e4 off by 5e-8 turns; a
// product carried from pair to pair 1e-7).  24 powers for 128 pairs, 0.15 us.
inline void rope_freq(double base, int rot, double* f) {
  double low[8];
  const int n = rot / 2;
  for (int j = 0; j < 8 && j < n; ++j) low[j] = pow(base, -2.0 * j / rot);
  for (int j = 0; j < n; j += 8) {
    const double high = 0.15915494309189533577 * pow(base, -2.0 * j / rot);   // 1 / (2 pi)
    for (int k = 0; k < 8 && j + k < n; ++k) f[j + k] = high * low[k];
  }
}

}  // namespace m3
