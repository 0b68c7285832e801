// How far a rotation turns a pair of columns at each position: theta^(-2c/r) / 2 pi, in 2^-64 of a turn.  Host code.
//
// A position of 2^31 leaves 2^-34 of a turn of an error of half a unit, and 2^-24.3 of a power in doubles (52 bits, times a
// rounded 1 / 2 pi: measured at theta 10^4, r 256).  So the numbers have 127 bits: a root in doubles, one Newton
// step, x <- x (1 - (theta x^n - 1) / n), and products.
#pragma once

#include <math.h>
#include <stdint.h>

namespace tv {

// m * 2^(e - 127), m in [2^126, 2^127)
struct Wide {
  unsigned __int128 m;
  int e;
};
inline Wide wide(double x) {  // x > 0, exact
  Wide w;
  w.m = (unsigned __int128)(uint64_t)ldexp(frexp(x, &w.e), 53) << 74;
  return w;
}
inline Wide settled(Wide x) {  // a bit at most past either end
  if (x.m >> 127) x.m >>= 1, ++x.e;
  if (!(x.m >> 126)) x.m <<= 1, --x.e;
  return x;
}
inline Wide product(Wide a, Wide b) {
  const unsigned __int128 a1 = a.m >> 64, a0 = (uint64_t)a.m, b1 = b.m >> 64, b0 = (uint64_t)b.m;
  const unsigned __int128 mid = a1 * b0 + a0 * b1 + (a0 * b0 >> 64);  // below 2^128: a1, b1 below 2^63
  return settled(Wide{(a1 * b1 << 1) + (mid >> 63), a.e + b.e});
}
// theta^(-1/n), good to 2^-95
inline Wide inverse_root(double theta, int n) {
  Wide x = wide(pow(theta, -1.0 / n)), y = wide(theta);
  for (int i = 0; i < n; ++i) y = product(y, x);
  // (y - 1) / n in 2^-126, below 2^-50: 1 is 2^126 with e = 1
  const __int128 off = ((__int128)(y.e == 1 ? y.m : y.m >> 1) - ((__int128)1 << 126)) / n;
  x.m -= (unsigned __int128)((__int128)(x.m >> 74) * (off >> 8) >> 44);  // x has 53 bits
  return settled(x);
}
// turns a position of the pairs c < rotary / 2
inline void turns_of(double theta, int rotary, unsigned long long* turns) {
  if (rotary == 0) return;
  const Wide step = inverse_root(theta, rotary / 2);
  Wide x{(unsigned __int128)0x517cc1b727220a94ull << 64 | 0xfe13abe8fa9a6ee0ull, -2};  // 1 / 2 pi
  for (int c = 0; c < rotary / 2; ++c, x = product(x, step)) {
    const int shift = 63 - x.e;
    turns[c] = shift > 127 ? 0 : (unsigned long long)(((x.m >> (shift - 1)) + 1) >> 1);
  }
}

}  // namespace tv
