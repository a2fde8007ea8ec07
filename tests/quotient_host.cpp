// spense_quotient.h on the host: every significand of a scale, with reciprocals
// that are a unit in the last place off, against the machine's own division.
#include "../sparse_dense_gemm_amd/csrc/spense_quotient.h"

#include <cstring>

using namespace spense;

namespace {
float of(uint32_t b) {
  float f;
  std::memcpy(&f, &b, 4);
  return f;
}
uint32_t bits(float f) {
  uint32_t b;
  std::memcpy(&b, &f, 4);
  return b;
}
}  // namespace

extern "C" {

int host_by_reciprocal(float s) { return by_reciprocal(s, bits(s)); }

// Whether r is within a unit in the last place of 1 / s (a double holds the
// difference well enough: no 1 / s is nearer than 2^-48 to such a border).
static bool near(float r, float s, float want) {
  const double unit = (double)of(bits(want) + 1u) - want;
  return fabs((double)r - 1.0 / (double)s) <= unit;
}

// Significands of scales 2^e (1 + m 2^-23), m = m0, m0 + step, ..., whose
// reciprocal comes out wrong from some start within a unit in the last place of
// 1 / s; with `all` those too that by_reciprocal turns away.  The first goes to
// *which.
int64_t host_wrong_reciprocals(int e, uint32_t m0, uint32_t step, int all, uint32_t* which) {
  int64_t wrong = 0;
  for (uint32_t m = m0; m < (1u << 23); m += step) {
    const float s = of(((uint32_t)(e + 127) << 23) | m);
    if (!all && !by_reciprocal(s, bits(s))) continue;
    const float want = 1.0f / s;
    for (int off = -1; off <= 1; ++off)
      if (near(of(bits(want) + (uint32_t)off), s, want) && reciprocal(s, of(bits(want) + (uint32_t)off)) != want) {
        if (!wrong++) *which = m;
        break;
      }
  }
  return wrong;
}

// The same of quotients x / s: x = borders[i] s and its neighbours up to two units.
int64_t host_wrong_quotients(int e, uint32_t m0, uint32_t step, const float* borders, int n, int all) {
  int64_t wrong = 0;
  for (uint32_t m = m0; m < (1u << 23); m += step) {
    const float s = of(((uint32_t)(e + 127) << 23) | m);
    if (!all && !by_reciprocal(s, bits(s))) continue;
    const float inv = 1.0f / s;
    for (int off = -1; off <= 1; ++off) {
      const float r = reciprocal(s, of(bits(inv) + (uint32_t)off));
      for (int i = 0; i < n; ++i)
        for (int d = -2; d <= 2; ++d) {
          const float x = of(bits(borders[i] * s) + (uint32_t)d);
          wrong += quotient(x, s, r) != x / s;
        }
    }
  }
  return wrong;
}

// x / 448 by the constant's reciprocal
int64_t host_wrong_scales(int e, uint32_t step) {
  int64_t wrong = 0;
  for (uint32_t m = 0; m < (1u << 23); m += step) {
    const float x = of(((uint32_t)(e + 127) << 23) | m);
    wrong += quotient(x, 448.0f, 1.0f / 448.0f) != x / 448.0f;
  }
  return wrong;
}

}  // extern "C"
