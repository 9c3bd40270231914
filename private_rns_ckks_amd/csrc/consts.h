// Real constants of a call as integers on the device: the host rounds them,
// kernels take them modulo each prime with their Shoup quotients.
#pragma once
#include <math.h>

#include "attention.h"

namespace ckks {

// m * 2^e: an integer next to a double.
struct Whole {
  int64_t m;
  int e;
};

// round(x), halves away from zero, for |x| < 2^126; false when out of range or
// not a number.  From 2^62 on x is an integer itself.
inline bool whole(double x, Whole* out) {
  if (!(fabs(x) < 0x1p126)) return false;
  if (fabs(x) < 0x1p62) {
    *out = Whole{(int64_t)llround(x), 0};
    return true;
  }
  int e;
  const double f = frexp(x, &e);  // 0.5 <= |f| < 1
  *out = Whole{(int64_t)ldexp(f, 53), e - 53};
  return true;
}

// What a scale has to be.
inline bool positive(double v) { return v > 0 && v < INFINITY; }

// The least integer for a constant that sets a result's scale: rounding moves it
// by 2^-20 of itself at most, what decrypted results are held to.
constexpr int64_t kLeastFactor = 1 << 19;
inline bool whole_factor(double x, Whole* out) { return whole(x, out) && out->m >= kLeastFactor; }

// A table of n constants for the limbs i < nl, limb by limb:
// table[(i * n + j) * 2] = {k_j mod q_i, Shoup quotient}.  With drop > 0, limbs
// i <= nl - 1 - drop hold k_j (q_(nl-1) .. q_(nl-drop))^-1 instead, which turns
// a product into the term that the rescales to come keep (DropOut).
struct ConstTable {
  const Whole* k;
  int n, nl, drop;
  uint64_t* table;  // const_words(n, nl)
};
inline uint64_t const_words(int n, int nl) { return (uint64_t)n * nl * 2; }
// All of a call's tables at once: few launches.
constexpr int kMaxConstTables = 8;
int launch_consts(Ctx* c, hipStream_t s, const ConstTable* t, int n_tables);

}  // namespace ckks
