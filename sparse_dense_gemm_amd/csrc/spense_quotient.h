// Quotients of fp32 numbers, rounded as a division rounds them, from a
// reciprocal and fused multiply-adds.  For the kernels, and for the host, where
// every significand can be tried.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace spense {

// The quotient x / d rounded to 32 bits, r = 1 / d rounded to nearest: two steps
// q += r (x - q d) in fused multiply-adds.  The first leaves q within a unit in the
// last place, the second's remainder is exact, and its sum rounds as the division
// does.  Five instructions where the division takes ten; it needs d, r and the
// remainders in the normal range.
__host__ __device__ __forceinline__ float quotient(float x, float d, float r) {
  float q = x * r;
  q = fmaf(fmaf(-q, d, x), r, q);
  return fmaf(fmaf(-q, d, x), r, q);
}

// 1 / s rounded to nearest, from r within a unit in the last place of it: one
// step.  Not for a significand of all ones, 1 / s then lying just above the middle
// between two numbers, where a step from below ends (or from two above).
__host__ __device__ __forceinline__ float reciprocal(float s, float r) { return fmaf(fmaf(-s, r, 1.0f), r, r); }

// Whether quotient(x, s, reciprocal(s, r)) has the e4m3 code of x / s for every
// |x| <= 449 s: s has room on both sides of it, so that only an x far below the
// smallest code can leave a remainder outside the normal range, and its significand
// is not all ones (one scale in 2^23).  The others divide.
__host__ __device__ __forceinline__ bool by_reciprocal(float s, uint32_t bits) {
  return s >= 0x1p-90f && s <= 0x1p100f && (bits & 0x7FFFFFu) != 0x7FFFFFu;
}

}  // namespace spense
