// mx_plan.h -- which form of the microscaled product a call takes.  Plain
// arithmetic on the call's sizes, compiled for the host by the library and by
// the check that every form is among the shapes that the tests multiply.
#pragma once

#include <cmath>
#include <cstdint>

namespace strata {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The form of a call, by what it costs: the stages that a CTA goes through
// (0.17 to 0.22 us each, most of it the issue of the scale copies and MMAs,
// so the tile's tokens count for little; half as much again where two CTAs
// share an SM), the join, reading the sums out.  The factors, in units of about
// 0.17 us, are fitted to every form's time on shapes of 1 to 1100 tokens, N to
// 24000, K to 8192 in all three pairs of formats.  On the 1238 of them that
// profiles/mx_linear_forms.csv lists this takes the best form, or one within 8 %
// of it, for 1227, and is 0.4 % behind on average.  Larger N is not fitted:
// past 5 tiles an SM calls of more than 64 tokens go to the pairs, half or more
// of whose 256 tokens are then padding (N = 128256, K = 4096, 8x4 bits: 64 us
// for 64 tokens, 85 for 65, 104 for 256).
// Measured, T = 4, 8x4 bits, with 1, 2, 4 and 8 ranks: N = 2560, K = 8192 15.9,
// 10.1, 7.5 and 6.7 us; N = 8192, K = 2048 6.5, 5.9 and 5.5 with 1, 2 and 4.
struct LinPlan {
  int nt, splits;  // tokens a tile, 0: the pairs' tiles; ranks a tile
};
inline LinPlan plan_linear(int T, int N, int K, bool f4, int num_sms) {
  // Tiles of 16 and 32 tokens are for calls with one: a tile starts at a
  // multiple of 64 (its scales at a tensor-memory column of their own).
  const int lo = T <= 16 ? 16 : T <= 32 ? 32 : 64, hi = T <= 64 ? lo : 128;
  const int chunks = (int)ceil_div(K, f4 ? 256 : 128);
  LinPlan best = {0, 1};
  double least = INFINITY;
  if (T > 32) {
    const double rounds = (double)ceil_div(ceil_div(T, 256) * ceil_div(N, 256), num_sms / 2);
    least = 12 + rounds * (chunks * (f4 ? 2.4 : 1.5) + 3);
  }
  for (int nt = lo; nt <= hi; nt *= 2) {
    const int64_t tiles = ceil_div(N, 128) * ceil_div(T, nt);
    if (T > 64 && tiles > 5 * num_sms) continue;  // (past what was fitted)
    for (int s = 1; s <= 8; s *= 2) {
      const int64_t ctas = tiles * s;
      // (the sums of 128 tokens twice over leave no room for a second CTA)
      if (s > 1 && (nt == 128 || ctas > 2 * num_sms || chunks < 2 * s)) break;
      const bool shared = ctas > num_sms;  // two CTAs an SM
      double cost = (double)ceil_div(chunks, s) * (f4 ? 1.5 : 1.0);
      if (shared) cost = (cost + 1.2) * (1.5 + 0.15 * nt / 64) * (double)ceil_div(ctas, 2 * num_sms);
      if (s > 1) cost += 0.2 + 0.14 * nt + (s == 8 && shared ? 1.4 : 0);
      cost += 0.09 * nt;
      if (cost < least) {
        least = cost;
        best = {nt, s};
      }
    }
  }
  return best;
}

// Of the pairs' tiles, those whose rows are turned in shared memory: they need
// rows of y on 16-byte boundaries, and are for calls of many rounds of tiles
// that take longer to multiply than to store.
inline bool plan_wide(int T, int N, int K, bool f4, bool aligned, int num_sms) {
  return aligned && ceil_div(T, 256) * ceil_div(N, 256) > 3 * (num_sms / 2) &&
         ceil_div(K, f4 ? 256 : 128) >= 8;
}

}  // namespace strata
