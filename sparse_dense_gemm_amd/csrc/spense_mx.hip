// HIP kernels of the microscaled 4-bit (mx4) format: quantisation,
// dequantisation and packing of weights (see spense_mx.h for the layouts).
//
// A block of 32 consecutive columns shares the power of two 2^(E - 127) with
//   E = clamp(floor(log2 max|x|) - 2 + 127, 0, 254), 0 for a block of zeros,
// so that the largest magnitude lands in [4, 8) and rounds to 4, 6 or (from 7
// on) saturates at 6; each code is the e2m1 number nearest to x 2^(127 - E),
// ties to the even code, the sign kept.  A block that holds a NaN or an
// infinity has E = 255 and zero codes.  All of it is exact: the maximum and its
// exponent field are integer operations, the scaling is by a power of two, and
// the conversion instruction rounds once.
#include "spense_device.h"
#include "spense_mx.h"

namespace spense {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
// vectors at any address (global loads and stores take any alignment): rows of
// odd lengths and matrices that start anywhere move at full width
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef uint32_t u32_any __attribute__((aligned(1)));

// exponent byte of a block whose largest magnitude has the fp32 bits `m`
__device__ __forceinline__ uint32_t block_exponent(uint32_t m) {
  if (m >= 0x7F800000u) return 255u;
  const uint32_t e = m >> 23;  // floor(log2) + 127 of a normal number
  // below 2^-124 (subnormals among them) floor(log2) - 2 + 127 is negative or zero
  return e > 2u ? e - 2u : 0u;
}

// 2^(E - 127) as fp32 bits (E < 255)
__device__ __forceinline__ float exponent_value(uint32_t e) { return __uint_as_float(e ? e << 23 : 0x00400000u); }

// the dword of eight codes of x / 2^(E - 127); zeros for a NaN block
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], uint32_t e) {
  if (e == 255u) return 0u;
  const float s = exponent_value(e);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[0], x[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], s, 3);
  return c;
}

// eight values of row x from column k on, zeros from K on
template <typename XT>
__device__ __forceinline__ void load8(const XT* x, int64_t k, int64_t K, float (&v)[8]) {
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

// Four lanes take a block, eight columns each: the maximum travels over the
// four lanes and each writes the four bytes of its codes.
// PACKED: the product kernel's activations (codes of 64 bytes per unit up to
// the last whole unit, exponent byte of unit 4 i + u, group g at 16 i + 4 g + u).
// Bound by memory: a lane reads 16 bytes of bf16 (2 x 16 of fp32) and writes
// four; 2048 x 27648 bf16 in 24.7 us, 5.8 TB/s (a copy reaches 5.0).  Rows of
// odd lengths and any alignment move in the same pieces (with dequantising, 59
// us instead of 145 by single elements).
template <typename XT, bool PACKED>
__global__ __launch_bounds__(256) void quantize_kernel(const XT* X, int64_t M, int64_t K, int64_t ldx,
                                                       const int32_t* rows, int64_t R, uint8_t* codes, int64_t ldc,
                                                       uint8_t* scales, int64_t lds, int64_t blocks) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;  // a launch has at most 2^30 threads
  const uint32_t b = id >> 2, brow = b / (uint32_t)blocks;
  const int64_t row = brow, col = b - brow * (uint32_t)blocks;
  const int q = (int)(id & 3);
  const bool in = row < R;
  const int64_t src = !in ? -1 : rows ? rows[row] : row;
  const int64_t k = col * kMxBlock + 8 * q;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (src >= 0 && src < M) load8<XT>(X + src * ldx, k, K, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7FFFFFFFu;
    m = u > m ? u : m;
  }
  uint32_t o = (uint32_t)__shfl_xor((int)m, 1);
  m = o > m ? o : m;
  o = (uint32_t)__shfl_xor((int)m, 2);
  m = o > m ? o : m;
  if (!in) return;
  const uint32_t e = block_exponent(m);
  const uint32_t c = codes8(v, e);
  if constexpr (PACKED) {
    const int64_t unit = col >> 2;
    if (unit < mx_units(K)) *(uint32_t*)(codes + row * ldc + col * 16 + 4 * q) = c;
    if (q == 0) scales[row * lds + (unit >> 2) * 16 + (col & 3) * 4 + (unit & 3)] = (uint8_t)e;
  } else {
    uint8_t* out = codes + row * ldc + col * 16 + 4 * q;
    const int64_t have = (K - k + 1) / 2;  // bytes of the row from here on
    if (have >= 4) {
      *(u32_any*)out = c;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < have) out[i] = (uint8_t)(c >> (8 * i));
    }
    if (q == 0) scales[row * lds + col] = (uint8_t)e;
  }
}

// Eight columns a thread, so that a bf16 result is one store of 16 bytes; bound
// by memory: 2048 x 27648 to bf16 in 23.0 us, 6.2 TB/s.
template <typename YT>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* codes, int64_t ldc, const uint8_t* scales,
                                                         int64_t lds, int64_t M, int64_t K, YT* Y, int64_t ldy) {
  const uint32_t per = (uint32_t)((K + 7) / 8), id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t r = id / per;
  const int64_t row = r, k = (int64_t)(id - r * per) * 8;
  if (row >= M) return;
  const uint8_t* in = codes + row * ldc + k / 2;
  uint32_t c = 0;
  const int64_t have = (K - k + 1) / 2;
  if (have >= 4) {
    c = *(const u32_any*)in;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) c |= (uint32_t)in[i] << (8 * i);
  }
  const uint32_t e = scales[row * lds + k / kMxBlock];
  const float s = e == 255u ? __uint_as_float(0x7FC00000u) : exponent_value(e);
  YT* out = Y + row * ldy + k;
  if constexpr (sizeof(YT) == 2) {
    u32x4 w;
    w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
    w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
    w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
    w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
    if (k + 8 <= K) {
      *(u32x4_any*)out = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) out[i] = (YT)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    f32x2 p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
    if (k + 8 <= K) {
      *(f32x4_any*)out = f32x4{p[0].x, p[0].y, p[1].x, p[1].y};
      *(f32x4_any*)(out + 4) = f32x4{p[2].x, p[2].y, p[3].x, p[3].y};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < K) out[i] = p[i / 2][i & 1];
    }
  }
}

// W row behind packed row r of an expert, -1 on padding rows
__device__ __forceinline__ int64_t packed_row(const ExpertsDesc& d, int64_t r) {
  if (!d.glu) return r < d.N ? r : -1;
  const int64_t I = d.N / 2, i = r >> 1;
  return i >= I ? -1 : (r & 1) * I + i;
}

// One thread per lane and unit (mx4) or lane, unit and step (bf16), 16 bytes
// each, of row tiles t0 .. t0 + tiles - 1 counted over the experts.  Runs once
// per weight matrix; its stores are whole units in order, its reads 16 bytes of
// a row.
template <bool MX>
__global__ __launch_bounds__(256) void pack_experts_kernel(ExpertsDesc d, int64_t t0, int64_t tiles, const uint8_t* W,
                                                           int64_t ldw) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;  // a launch has at most 2^30 threads
  const int lane = (int)(id & 63);
  const uint32_t per = (uint32_t)(MX ? d.NU : 4 * d.NU);  // kilobytes of a row tile
  const uint32_t kb = id >> 6, i = kb / per, u = kb - i * per;
  if (i >= tiles) return;
  const int64_t tile = t0 + i;
  const int64_t e = tile / d.NT, rt = tile - e * d.NT;
  const int64_t src = packed_row(d, rt * 16 + (lane & 15));
  const int g = lane >> 4;
  union {
    uint8_t b[16];
    uint16_t h[8];
    u32x4 v;
  } o;
  o.v = u32x4{0, 0, 0, 0};
  if (src >= 0) {
    if constexpr (MX) {
      const int64_t k = (int64_t)u * kUnitK + 32 * g;
      const uint8_t* w = W + (e * d.N + src) * ldw + k / 2;
      if (k + 32 <= d.K) {
        o.v = *(const u32x4_any*)w;
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (k + 2 * q + 1 < d.K) o.b[q] = w[q];
          else if (k + 2 * q < d.K) o.b[q] = w[q] & 15;
        }
      }
    } else {
      const int64_t k = (int64_t)u * 32 + 8 * g;
      const uint16_t* w = (const uint16_t*)W + (e * d.N + src) * ldw + k;
      if (k + 8 <= d.K) {
        o.v = *(const u32x4_any*)w;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (k + q < d.K) o.h[q] = w[q];
      }
    }
  }
  *(u32x4*)(d.wpack + tile * d.tile_bytes + (int64_t)u * 1024 + lane * 16) = o.v;
}

// One thread per lane and four units: their exponent bytes.
__global__ __launch_bounds__(256) void pack_exponents_kernel(ExpertsDesc d, int64_t t0, int64_t tiles,
                                                             const uint8_t* scales, int64_t lds) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const int lane = (int)(id & 63);
  const uint32_t per = (uint32_t)((d.NU + 3) / 4);
  const uint32_t q = id >> 6, i = q / per, i4 = q - i * per;
  if (i >= tiles) return;
  const int64_t tile = t0 + i;
  const int64_t e = tile / d.NT, rt = tile - e * d.NT;
  const int64_t src = packed_row(d, rt * 16 + (lane & 15));
  uint32_t o = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t b = (4 * (int64_t)i4 + u) * 4 + (lane >> 4);  // block of 32 columns
    const uint32_t v = src >= 0 && b * kMxBlock < d.K ? scales[(e * d.N + src) * lds + b] : 127u;
    o |= v << (8 * u);
  }
  *(uint32_t*)(d.wpack + tile * d.tile_bytes + d.scale_off + (int64_t)i4 * 256 + lane * 4) = o;
}

unsigned groups(int64_t threads) { return (unsigned)((threads + 255) / 256); }

// A launch's grid counts threads in 32 bits: f(first row, rows) over runs of
// rows of at most 2^30 threads (a row takes at most 2^18, a row tile of weights
// in packing at most 2^21).
template <typename F>
hipError_t by_rows(int64_t rows, int64_t threads_per_row, F&& f) {
  const int64_t most = (int64_t(1) << 30) / threads_per_row;
  for (int64_t r = 0; r < rows; r += most) {
    f(r, rows - r < most ? rows - r : most);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool PACKED>
hipError_t quantize(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R,
                    uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s) {
  const int64_t blocks = PACKED ? (mx_units(K) + 3) / 4 * 16 : (K + kMxBlock - 1) / kMxBlock;
  return by_rows(R, blocks * 4, [&](int64_t r0, int64_t n) {
    // rows picked by index keep X's origin
    const int64_t x0 = rows ? 0 : r0 * ldx;
    const int32_t* pick = rows ? rows + r0 : nullptr;
    const int64_t have = rows ? M : n;
    if (xdtype == DT_F32)
      quantize_kernel<float, PACKED><<<groups(n * blocks * 4), 256, 0, s>>>(
          (const float*)X + x0, have, K, ldx, pick, n, codes + r0 * ldc, ldc, scales + r0 * lds, lds, blocks);
    else
      quantize_kernel<uint16_t, PACKED><<<groups(n * blocks * 4), 256, 0, s>>>(
          (const uint16_t*)X + x0, have, K, ldx, pick, n, codes + r0 * ldc, ldc, scales + r0 * lds, lds, blocks);
  });
}

}  // namespace

hipError_t launch_mx4_quantize(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                               int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s) {
  return quantize<false>(X, xdtype, M, K, ldx, nullptr, M, codes, ldc, scales, lds, s);
}

hipError_t launch_mx4_activations(const void* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R,
                                  uint8_t* codes, int64_t ldc, uint8_t* scales, int64_t lds, hipStream_t s) {
  return quantize<true>(X, DT_BF16, M, K, ldx, rows, R, codes, ldc, scales, lds, s);
}

hipError_t launch_mx4_dequantize(const uint8_t* codes, int64_t ldc, const uint8_t* scales, int64_t lds, int64_t M,
                                 int64_t K, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s) {
  const int64_t per = (K + 7) / 8;
  return by_rows(M, per, [&](int64_t r0, int64_t n) {
    if (ydtype == DT_F32)
      dequantize_kernel<float><<<groups(n * per), 256, 0, s>>>(codes + r0 * ldc, ldc, scales + r0 * lds, lds, n, K,
                                                               (float*)Y + r0 * ldy, ldy);
    else
      dequantize_kernel<uint16_t><<<groups(n * per), 256, 0, s>>>(codes + r0 * ldc, ldc, scales + r0 * lds, lds, n, K,
                                                                  (uint16_t*)Y + r0 * ldy, ldy);
  });
}

hipError_t launch_pack_experts(const ExpertsDesc& d, const void* W, int64_t ldw, const uint8_t* scales, int64_t lds,
                               hipStream_t s) {
  const bool mx = d.wdtype == DT_MX4;
  const int64_t per = d.NU * (mx ? 64 : 256), per4 = (d.NU + 3) / 4 * 64;
  return by_rows(d.E * d.NT, per, [&](int64_t t0, int64_t n) {
    if (mx) {
      pack_experts_kernel<true><<<groups(n * per), 256, 0, s>>>(d, t0, n, (const uint8_t*)W, ldw);
      pack_exponents_kernel<<<groups(n * per4), 256, 0, s>>>(d, t0, n, scales, lds);
    } else {
      pack_experts_kernel<false><<<groups(n * per), 256, 0, s>>>(d, t0, n, (const uint8_t*)W, ldw);
    }
  });
}

}  // namespace spense
