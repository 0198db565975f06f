// Rotation frequencies as fractions of a turn in 64-bit fixed point:
//   F_i = 2^64 (theta^(-2i/D) / (2 pi) modulo 1),
// so that position * F_i modulo 2^64 is the angle of any position below 2^31, off by less than
// 2^-29 of a turn (2^-32 for theta >= 1). That takes F_i to 64 places behind the point, and for
// theta < 1 as many more before it: more than a double (or an x86 long double) holds. Here a
// number is 128 bits and an exponent, in whole-number arithmetic, which gives the same table on
// every host.
//
// D / 2 is a power of two, 2^k, so theta^(-2/D) is k square roots of 1 / theta; the powers follow
// by multiplication. An inverse square root is Newton's iteration y <- y (3 - x y^2) / 2 from a
// double's: 52 good bits become 104, then all. A product is off by 2^-126 of its value, a root by
// 2^-123; after at most 255 products F_i is good to 2^-114, which is why theta is at least 2^-56:
// fewer than 2^54 turns a position, 2^31 positions, and 2^-29 of a turn is left.
#pragma once

#include <cmath>
#include <cstdint>

namespace pkv {

constexpr float kLeastTheta = 0x1p-56f;

namespace turns {

using u128 = unsigned __int128;

// m * 2^(e - 128), m's top bit set
struct Wide {
  u128 m;
  int e;
};

inline Wide wide(double x) {   // x > 0
  int e;
  const double f = std::frexp(x, &e);
  return {static_cast<u128>(static_cast<uint64_t>(std::ldexp(f, 64))) << 64, e};
}

inline Wide times(const Wide &a, const Wide &b) {
  const uint64_t ah = static_cast<uint64_t>(a.m >> 64), al = static_cast<uint64_t>(a.m);
  const uint64_t bh = static_cast<uint64_t>(b.m >> 64), bl = static_cast<uint64_t>(b.m);
  const u128 hl = static_cast<u128>(ah) * bl, lh = static_cast<u128>(al) * bh;
  const u128 ll = static_cast<u128>(al) * bl;
  const u128 mid = (ll >> 64) + static_cast<uint64_t>(hl) + static_cast<uint64_t>(lh);
  Wide r = {static_cast<u128>(ah) * bh + (hl >> 64) + (lh >> 64) + (mid >> 64), a.e + b.e};
  if (!(r.m >> 127)) {   // (a bit of what was cut off moves up)
    r.m = r.m << 1 | (static_cast<uint64_t>(mid) >> 63);
    --r.e;
  }
  return r;
}

inline Wide inverse_root(const Wide &x) {
  Wide y = wide(1.0 / std::sqrt(std::ldexp(static_cast<double>(static_cast<uint64_t>(x.m >> 64)),
                                           x.e - 64)));
  for (int i = 0; i < 3; ++i) {
    const Wide t = times(times(x, y), y);   // near 1: its exponent is 0 or 1
    // (3 - t) / 2, near 1, in units of 2^-127
    Wide w = {(static_cast<u128>(3) << 126) - (t.m >> (2 - t.e)), 1};
    if (!(w.m >> 127)) w.m <<= 1, w.e = 0;
    y = times(y, w);
  }
  return y;
}

// the places behind the point, 64 of them
inline uint64_t fraction(const Wide &x) {
  if (x.e > 64) return static_cast<uint64_t>(x.m << (x.e - 64));
  return x.e <= -64 ? 0 : static_cast<uint64_t>(x.m >> (64 - x.e));
}

}  // namespace turns

// f[i] = F_i for i < pairs (at most D / 2); theta finite, at least kLeastTheta
inline void rotation_turns(float theta, int pairs, int D, uint64_t *f) {
  using namespace turns;
  Wide step = inverse_root(wide(theta));   // theta^(-1/2)
  for (int d = 4; d < D; d *= 2) step = times(step, inverse_root(step));
  Wide x = {static_cast<u128>(0xa2f9836e4e441529ull) << 64 | 0xfc2757d1f534ddc0ull, -2};
  for (int i = 0; i < pairs; ++i) {        // x: 1 / (2 pi), and on
    f[i] = fraction(x);
    x = times(x, step);
  }
}

}  // namespace pkv
