// Device helpers of the block-scaled e4m3 format: the scale of a block, codes
// of eight values, eight values of a row.  Inline and file-local to each
// translation unit that includes it.
#pragma once

#include "spense_device.h"
#include "spense_fp8b.h"
#include "spense_quotient.h"

namespace spense {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
// vectors at any address (global loads and stores take any alignment)
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// two fp32 as bf16, rounded to nearest even
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// The scale of a block whose largest magnitude has the fp32 bits `m`: the
// quotient by 448, 1 where that is 0, NaN for a block that holds a NaN or an
// infinity.
__device__ __forceinline__ float block_scale(uint32_t m) {
  const float x = __uint_as_float(m);
  if (m >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  if (x >= 0x1p-80f) return quotient(x, kFp8Top, 1.0f / kFp8Top);
  const float s = x / kFp8Top;
  return s > 0.f ? s : 1.0f;
}

// The codes of four values of a block: e4m3(x / s), x / s being the 32-bit
// quotient (2048 x 27648 bf16 is bound by memory also with a division, but its
// vector instructions then take 29 instead of 17 us of 34).  Scales outside
// [2^-90, 2^100], and those whose significand is all ones, divide.
__device__ __forceinline__ uint32_t codes4(const f32x4& x, float s) {
  f32x4 q;
  if (by_reciprocal(s, __float_as_uint(s))) {
    const float r = reciprocal(s, __builtin_amdgcn_rcpf(s));
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __builtin_copysignf(quotient(x[i], s, r), x[i]);  // -0 stays
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = x[i] / s;
  }
  // a rounded scale may leave the largest quotient above 448
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_fmed3f(q[i], -kFp8Top, kFp8Top);
  int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  c = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], c, true);
  return s == s ? (uint32_t)c : 0u;
}
__device__ __forceinline__ u32x2 codes8(const float (&x)[8], float s) {
  return u32x2{codes4(f32x4{x[0], x[1], x[2], x[3]}, s), codes4(f32x4{x[4], x[5], x[6], x[7]}, s)};
}

// largest magnitude, as fp32 bits
__device__ __forceinline__ uint32_t top_of(const f32x4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = u > m ? u : m;
  }
  return m;
}
__device__ __forceinline__ uint32_t top8(const float (&v)[8]) {
  const uint32_t a = top_of(f32x4{v[0], v[1], v[2], v[3]}), b = top_of(f32x4{v[4], v[5], v[6], v[7]});
  return a > b ? a : b;
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
  // the loads go out together: no branch around one
  XT u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = x[k + i < K ? k + i : K - 1];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f;
    if constexpr (sizeof(XT) == 2) f = __uint_as_float((uint32_t)u[i] << 16);
    else f = u[i];
    v[i] = k + i < K ? f : 0.f;
  }
}

// Stores of whole pieces.  STREAM: with the non-temporal hint, for results larger
// than the caches that their next reader could find them in.
template <bool STREAM>
__device__ __forceinline__ void store_piece(u32x2_any* p, const u32x2& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool STREAM>
__device__ __forceinline__ void store_piece(u32x4_any* p, const u32x4& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <bool STREAM>
__device__ __forceinline__ void store_piece(f32x4_any* p, const f32x4& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// eight values of a row into fp32 or bf16 (rounded to nearest even), up to column K
template <bool STREAM, typename YT>
__device__ __forceinline__ void store_row8(YT* y, int64_t k, int64_t K, const float (&v)[8]) {
  if (k + 8 <= K) {
    if constexpr (sizeof(YT) == 2) {
      u32x4 u;
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
      store_piece<STREAM>((u32x4_any*)(y + k), u);
    } else {
      store_piece<STREAM>((f32x4_any*)(y + k), f32x4{v[0], v[1], v[2], v[3]});
      store_piece<STREAM>((f32x4_any*)(y + k + 4), f32x4{v[4], v[5], v[6], v[7]});
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
template <bool STREAM>
__device__ __forceinline__ void store_codes8(uint8_t* y, int64_t k, int64_t K, const u32x2& c) {
  if (k + 8 <= K) {
    store_piece<STREAM>((u32x2_any*)(y + k), c);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (k + i < K) y[k + i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
}

// Bytes of results from which on they are streamed: what the eight L2 caches hold.
// (quantise 25600 x 5120 fp32 and back, 131 + 262 MB out: 179 us, 199 without;
// below it a product that reads 10 MB of codes right after them finds them there)
constexpr int64_t kStreamBytes = int64_t(32) << 20;

}  // namespace
}  // namespace spense
