// gq_range.h -- which coefficients of the orthogonalised update keep its numbers within the range of the
// products' operands (host code, without HIP).
#pragma once

#include <stdint.h>

#include <cmath>
#include <initializer_list>

namespace gq {

// Whether singular values that begin in [0, 1] stay in the range of the products' operands: the
// largest |p(x)| = |a x + b x^3 + c x^5| on [0, top] lies at top or where a + 3 b x^2 + 5 c x^4 = 0,
// the largest |b x + c x^2| on [0, top^2] at top^2 or at -b / 2c.
//
// Each step's roundings may carry a value past the largest |p|, from where the next one may go anywhere:
// the interval is widened by them.  An operand in halves is off by 2^-11 at most.  A = X X^T has the roundings
// of X twice, and those of its own halves: 3 * 2^-11 top^2.  B = b A + c A^2 takes a change of A to at most
// |b + c (l + l')| of it, l and l' in [0, top^2], a linear function, and has roundings of its own, 2^-11 |B|;
// and B X has X's once more.
inline bool ortho_stays(int32_t steps, double a, double b, double c) {
  auto p = [&](double x) { return std::fabs(x * (a + x * x * (b + x * x * c))); };
  auto q = [&](double x) { return std::fabs(x * (b + x * c)); };
  double top = 1.0;
  for (int32_t i = 0; i < steps; ++i) {
    const double square = top * top;
    double most = p(top), off = q(square);
    if (c != 0.0 && -b / (2.0 * c) > 0.0 && -b / (2.0 * c) < square) off = std::fmax(off, q(-b / (2.0 * c)));
    const double d = 9.0 * b * b - 20.0 * a * c;
    if (d >= 0.0) {
      // both roots without a difference of near numbers, whatever c is; a root that is not there comes
      // out as an infinity or NaN
      const double sum = -0.5 * (3.0 * b + std::copysign(std::sqrt(d), b));
      for (double root : {sum / (5.0 * c), a / sum})
        if (root > 0.0 && root < square) most = std::fmax(most, p(std::sqrt(root)));
    }
    most += 0x1p-11 * top * (3.0 * square * std::fmax(std::fabs(b), std::fabs(b + 2.0 * c * square)) + 2.0 * off);
    if (!(most <= 7.5) || !(off <= 60.0)) return false;
    top = most;
  }
  return true;
}

}  // namespace gq
