// Device helpers of the block-scaled e4m3 format: the scale of a block, codes
// of eight values, eight values of a row.  Inline and file-local to each
// translation unit that includes it.
#pragma once

#include "spense_device.h"
#include "spense_fp8b.h"

namespace spense {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
// vectors at any address (global loads and stores take any alignment)
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// The scale of a block whose largest magnitude has the fp32 bits `m`: the
// quotient by 448, 1 where that is 0, NaN for a block that holds a NaN or an
// infinity.
__device__ __forceinline__ float block_scale(uint32_t m) {
  if (m >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  const float s = __uint_as_float(m) / kFp8Top;
  return s > 0.f ? s : 1.0f;
}

// The codes of eight values of a block: e4m3(x / s), x / s being the 32-bit
// quotient.  With r = 1 / s rounded once, two steps q += r (x - q s) in fused
// multiply-adds give that quotient: the first leaves it within a unit in the last
// place, the second is exact in its remainder and rounds as the division does
// (five instructions where the division takes ten; 2048 x 27648 bf16 is bound by
// memory with either, its vector instructions take 17 or 29 us of 34).  That
// needs s and the remainders in the normal range; the scales outside [2^-90,
// 2^100] divide.
__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float s) {
  float q[8];
  if (s >= 0x1p-90f && s <= 0x1p100f) {
    const float r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = x[i] * r;
      v = fmaf(fmaf(-v, s, x[i]), r, v);
      v = fmaf(fmaf(-v, s, x[i]), r, v);
      q[i] = __builtin_copysignf(v, x[i]);  // -0 stays
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = x[i] / s;
  }
  // a rounded scale may leave the largest quotient above 448
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_fmed3f(q[i], -kFp8Top, kFp8Top);
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  return s == s ? u32x2{(uint32_t)lo, (uint32_t)hi} : u32x2{0u, 0u};
}

// largest magnitude of eight values, as fp32 bits
__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = u > m ? u : m;
  }
  return m;
}

// the largest of m over the 16 lanes of a row (row rotations)
__device__ __forceinline__ uint32_t row_max(uint32_t m) {
  auto take = [&](int o) { m = (uint32_t)o > m ? (uint32_t)o : m; };
  take(__builtin_amdgcn_update_dpp(0, (int)m, 0x128, 0xF, 0xF, false));
  take(__builtin_amdgcn_update_dpp(0, (int)m, 0x124, 0xF, 0xF, false));
  take(__builtin_amdgcn_update_dpp(0, (int)m, 0x122, 0xF, 0xF, false));
  take(__builtin_amdgcn_update_dpp(0, (int)m, 0x121, 0xF, 0xF, false));
  return m;
}

// eight values of a row (fp32 or bf16) from column k on, zeros from K on
template <typename XT>
__device__ __forceinline__ void load_row8(const XT* x, int64_t k, int64_t K, float (&v)[8]) {
  if (k + 8 <= K) {
    if constexpr (sizeof(XT) == 2) {
      const u32x4 u = *(const u32x4_any*)(x + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
      const f32x4 a = *(const f32x4_any*)(x + k), b = *(const f32x4_any*)(x + k + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = 0.f;
    if (k + i < K) {
      if constexpr (sizeof(XT) == 2) v[i] = __uint_as_float((uint32_t)x[k + i] << 16);
      else v[i] = x[k + i];
    }
  }
}

// eight values of a row into fp32 or bf16 (rounded to nearest even), up to column K
template <typename YT>
__device__ __forceinline__ void store_row8(YT* y, int64_t k, int64_t K, const float (&v)[8]) {
  if (k + 8 <= K) {
    if constexpr (sizeof(YT) == 2) {
      typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
      u32x4 u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf16x2 p;
        p[0] = (__bf16)v[2 * i];
        p[1] = (__bf16)v[2 * i + 1];
        u[i] = __builtin_bit_cast(uint32_t, p);
      }
      *(u32x4_any*)(y + k) = u;
    } else {
      *(f32x4_any*)(y + k) = f32x4{v[0], v[1], v[2], v[3]};
      *(f32x4_any*)(y + k + 4) = f32x4{v[4], v[5], v[6], v[7]};
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) {
      if constexpr (sizeof(YT) == 2) y[k + i] = (YT)bf16_rne(v[i]);
      else y[k + i] = v[i];
    }
}

// eight codes of a row, up to column K
__device__ __forceinline__ void store_codes8(uint8_t* y, int64_t k, int64_t K, const u32x2& c) {
  if (k + 8 <= K) {
    *(u32x2_any*)(y + k) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) y[k + i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
}

}  // namespace
}  // namespace spense
