// HIP kernels of the block-scaled e4m3 format (fp8b): quantisation,
// dequantisation, packing of weights and the product's activations (see
// spense_fp8b.h for the layouts).
//
//   s = max|x| / 448 over the block (1 where that is 0),  code = e4m3(x / s),
// both quotients rounded to 32 bits, the code to nearest even; a block that
// holds a NaN or an infinity has a NaN for its scale and codes 0.
#include "spense_fp8b_device.h"

namespace spense {
namespace {

constexpr int kLanes = kFp8Block / 8;  // lanes of a block's row, eight columns each

// A scale for 128 columns of a row: sixteen lanes take a block, eight columns
// each; the maximum travels over them by row rotations.
// PADDED: the product kernel's activations (codes 0 from K to whole units).
// Bound by memory: a lane reads 16 bytes of bf16 (2 x 16 of fp32), writes eight;
// 2048 x 27648 bf16 in 34 us, 171 MB at 5.0 TB/s; one row of 5120 in 2.0 us.
template <typename XT, bool PADDED, bool STREAM>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const XT* X, int64_t M, int64_t K, int64_t ldx,
                                                            const int32_t* rows, int64_t R, uint8_t* codes,
                                                            int64_t ldc, float* scales, int64_t lds, uint32_t blocks) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;  // a launch has at most 2^30 threads
  const uint32_t b = id / kLanes, row = b / blocks, col = b - row * blocks;
  const bool in = row < R;
  const int64_t src = !in ? -1 : rows ? rows[row] : (int64_t)row;
  const int64_t k = (int64_t)col * kFp8Block + 8 * (id % kLanes);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (src >= 0 && src < M) load_row8<XT>(X + src * ldx, k, K, v);
  const float s = block_scale(row_max(top8(v)));
  if (!in) return;
  const u32x2 c = codes8(v, s);
  uint8_t* out = codes + (int64_t)row * ldc;
  if constexpr (PADDED) *(u32x2*)(out + k) = c;
  else store_codes8<STREAM>(out, k, K, c);
  if (id % kLanes == 0) scales[(int64_t)row * lds + col] = s;
}

// A scale for 128 rows x 128 columns: a workgroup takes a block, a wave four of
// its rows at a time, so that the block is read once and kept in registers while
// its maximum goes through LDS.  Bound by memory: 25600 x 5120 fp32 in 110 us,
// 655 MB at 6.0 TB/s.
template <typename XT, bool STREAM>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const XT* X, int64_t M, int64_t K, int64_t ldx,
                                                              uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                                                              uint32_t blocks) {
  __shared__ uint32_t top[4];
  const uint32_t brow = blockIdx.x / blocks, bcol = blockIdx.x - brow * blocks;
  const int64_t r0 = (int64_t)brow * kFp8Block + threadIdx.x / kLanes;
  const int64_t k = (int64_t)bcol * kFp8Block + 8 * (threadIdx.x % kLanes);
  constexpr int kPer = kFp8Block * kLanes / 256;  // rows of a thread, 16 apart
  float v[kPer][8];
  uint32_t m = 0;
  // past the last row that row again, which changes no maximum: all rows' loads go
  // out together
  auto load = [&](int64_t end) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) load_row8<XT>(X + (r0 + 16 * i < M ? r0 + 16 * i : M - 1) * ldx, k, end, v[i]);
  };
  if (k + 8 <= K) load(k + 8);
  else load(K);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint32_t t = top8(v[i]);
    m = t > m ? t : m;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t t = (uint32_t)__shfl_xor((int)m, o);
    m = t > m ? t : m;
  }
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) m = top[i] > m ? top[i] : m;
  const float s = block_scale(m);
  if (threadIdx.x == 0) scales[(int64_t)brow * lds + bcol] = s;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t r = r0 + 16 * i;
    if (r < M) store_codes8<STREAM>(codes + r * ldc, k, K, codes8(v[i], s));
  }
}

// Eight columns a thread: one store of 16 bytes of bf16 (two of fp32).  Bound by
// memory: 25600 x 5120 into bf16 in 66 us, 393 MB at 6.0 TB/s.
template <typename YT, bool STREAM>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint8_t* codes, int64_t ldc, const float* scales,
                                                         int64_t lds, int rows, int64_t M, int64_t K, YT* Y,
                                                         int64_t ldy) {
  const uint32_t per = (uint32_t)((K + 7) / 8), id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t r = id / per;
  const int64_t row = r, k = (int64_t)(id - r * per) * 8;
  if (row >= M) return;
  const uint8_t* in = codes + row * ldc + k;
  u32x2 c = u32x2{0u, 0u};
  if (k + 8 <= K) {
    c = *(const u32x2_any*)in;
  } else {
    uint8_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = in[k + i < K ? i : 0];  // no branch around a load
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i >> 2] |= (k + i < K ? (uint32_t)u[i] : 0u) << (8 * (i & 3));
  }
  const float s = scales[row / rows * lds + k / kFp8Block];
  float v[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[h], true);
    v[4 * h] = a.x * s;
    v[4 * h + 1] = a.y * s;
    v[4 * h + 2] = b.x * s;
    v[4 * h + 3] = b.y * s;
  }
  store_row8<STREAM>(Y + row * ldy, k, K, v);
}

// Codes and scales that are there already as the product kernel reads them:
// rows of whole units (codes 0 from K on), picked by index if asked for.  Sixteen
// codes a thread (2048 x 5120: 6.6 us, 21 MB).
__global__ __launch_bounds__(256) void lay_out_kernel(const uint8_t* X, int64_t ldx, const float* sx, int64_t lds_in,
                                                      int64_t M, int64_t K, const int32_t* rows, int64_t R,
                                                      uint8_t* codes, int64_t ldc, float* scales, int64_t lds) {
  const uint32_t per = (uint32_t)(ldc / 16), id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t r = id / per;
  if (r >= R) return;
  const int64_t row = r, k = (int64_t)(id - r * per) * 16;
  const int64_t src = rows ? rows[row] : row;
  const bool in = src >= 0 && src < M;
  u32x4 o = u32x4{0, 0, 0, 0};
  if (in && k + 16 <= K) {
    o = *(const u32x4_any*)(X + src * ldx + k);
  } else if (in) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (k + i < K) o[i >> 2] |= (uint32_t)X[src * ldx + k + i] << (8 * (i & 3));
  }
  *(u32x4*)(codes + row * ldc + k) = o;
  if (k % kFp8Block == 0) scales[row * lds + k / kFp8Block] = in ? sx[src * lds_in + k / kFp8Block] : 0.f;
}

// W row behind packed row r of an expert, -1 on padding rows
__device__ __forceinline__ int64_t packed_row(const Fp8bDesc& d, int64_t r) {
  if (!d.glu) return r < d.N ? r : -1;
  const int64_t I = d.N / 2, i = r >> 1;
  return i >= I ? -1 : (r & 1) * I + i;
}

// One thread per 16-byte piece of row tiles t0 .. t0 + tiles - 1 counted over
// the experts.  Runs once per weight matrix (25600 x 5120: 41 us); its stores are
// whole kilobytes.
__global__ __launch_bounds__(256) void pack_kernel(Fp8bDesc d, int64_t t0, int64_t tiles, const uint8_t* W,
                                                   int64_t ldw) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const int lane = (int)(id & 63);
  const uint32_t per = (uint32_t)(2 * d.NU);  // kilobytes of a row tile
  const uint32_t kb = id >> 6, i = kb / per, u = kb - i * per;
  if (i >= tiles) return;
  const int64_t tile = t0 + i;
  const int64_t e = tile / d.NT, rt = tile - e * d.NT;
  const int64_t src = packed_row(d, rt * 16 + (lane & 15));
  const int64_t k = (int64_t)(u >> 1) * kUnitK + 64 * (u & 1) + 16 * (lane >> 4);
  u32x4 o = u32x4{0, 0, 0, 0};
  if (src >= 0) {
    const uint8_t* w = W + (e * d.N + src) * ldw + k;
    if (k + 16 <= d.K) {
      o = *(const u32x4_any*)w;
    } else {
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (k + q < d.K) o[q >> 2] |= (uint32_t)w[q] << (8 * (q & 3));
    }
  }
  *(u32x4*)(d.wpack + tile * d.tile_bytes + (int64_t)u * 1024 + lane * 16) = o;
}

// One thread per scale of groups g0 .. g0 + groups - 1 counted over the experts.
__global__ __launch_bounds__(256) void pack_scales_kernel(Fp8bDesc d, int64_t g0, int64_t groups, const float* scales,
                                                          int64_t lds) {
  const uint32_t id = blockIdx.x * 256u + threadIdx.x;
  const uint32_t per = (uint32_t)(2 * d.NUe), i = id / per, j = id - i * per;
  if (i >= groups) return;
  const int64_t grp = g0 + i, e = grp / d.SG, g = grp - e * d.SG;
  const int64_t u = j >> 1, odd = j & 1;
  float s = 0.f;
  if (u < d.NU) {
    if (d.glu) {
      const int64_t nb = (d.N / 2 + kFp8Block - 1) / kFp8Block;  // blocks of the gate, and of up
      s = scales[(e * 2 * nb + odd * nb + g / 2) * lds + u];     // 128 packed rows: 64 of each
    } else {
      s = scales[(e * d.SG + g) * lds + u];
    }
  }
  d.scales[grp * per + j] = s;
}

unsigned groups_of(int64_t threads) { return (unsigned)((threads + 255) / 256); }

// A launch's grid counts threads in 32 bits: f(first row, rows) over runs of
// rows of at most 2^30 threads (a row takes at most 2^24).
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

template <bool PADDED, bool STREAM, typename XT>
void quantize_rows(const XT* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R, uint8_t* codes,
                   int64_t ldc, float* scales, int64_t lds, hipStream_t s) {
  const int64_t blocks = (K + kFp8Block - 1) / kFp8Block;
  quantize_rows_kernel<XT, PADDED, STREAM><<<groups_of(R * blocks * kLanes), 256, 0, s>>>(
      X, M, K, ldx, rows, R, codes, ldc, scales, lds, (uint32_t)blocks);
}

template <bool STREAM, typename XT>
hipError_t quantize(const XT* X, int64_t M, int64_t K, int64_t ldx, int rows, uint8_t* codes, int64_t ldc,
                    float* scales, int64_t lds, hipStream_t s) {
  const int64_t blocks = (K + kFp8Block - 1) / kFp8Block;
  if (rows == 1)
    return by_rows(M, blocks * kLanes, [&](int64_t r0, int64_t n) {
      quantize_rows<false, STREAM>(X + r0 * ldx, n, K, ldx, nullptr, n, codes + r0 * ldc, ldc, scales + r0 * lds, lds, s);
    });
  return by_rows((M + rows - 1) / rows, blocks * 256, [&](int64_t b0, int64_t n) {
    const int64_t r0 = b0 * rows, m = M - r0 < n * rows ? M - r0 : n * rows;
    quantize_blocks_kernel<XT, STREAM><<<(unsigned)(n * blocks), 256, 0, s>>>(
        X + r0 * ldx, m, K, ldx, codes + r0 * ldc, ldc, scales + b0 * lds, lds, (uint32_t)blocks);
  });
}

template <bool STREAM, typename YT>
hipError_t dequantize(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int rows, int64_t M,
                      int64_t K, YT* Y, int64_t ldy, hipStream_t s) {
  const int64_t per = (K + 7) / 8;
  // runs of whole blocks of rows
  return by_rows((M + kFp8Block - 1) / kFp8Block, per * kFp8Block, [&](int64_t b0, int64_t n) {
    const int64_t r0 = b0 * kFp8Block, m = M - r0 < n * kFp8Block ? M - r0 : n * kFp8Block;
    dequantize_kernel<YT, STREAM><<<groups_of(m * per), 256, 0, s>>>(codes + r0 * ldc, ldc, scales + r0 / rows * lds, lds,
                                                                     rows, m, K, Y + r0 * ldy, ldy);
  });
}

}  // namespace

hipError_t launch_fp8b_quantize(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, int rows,
                                uint8_t* codes, int64_t ldc, float* scales, int64_t lds, hipStream_t s) {
  const bool stream = M * K > kStreamBytes;
  if (xdtype == DT_F32)
    return stream ? quantize<true>((const float*)X, M, K, ldx, rows, codes, ldc, scales, lds, s)
                  : quantize<false>((const float*)X, M, K, ldx, rows, codes, ldc, scales, lds, s);
  return stream ? quantize<true>((const uint16_t*)X, M, K, ldx, rows, codes, ldc, scales, lds, s)
                : quantize<false>((const uint16_t*)X, M, K, ldx, rows, codes, ldc, scales, lds, s);
}

hipError_t launch_fp8b_dequantize(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int rows,
                                  int64_t M, int64_t K, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s) {
  const bool f32 = ydtype == DT_F32, stream = M * K * (f32 ? 4 : 2) > kStreamBytes;
  if (f32)
    return stream ? dequantize<true>(codes, ldc, scales, lds, rows, M, K, (float*)Y, ldy, s)
                  : dequantize<false>(codes, ldc, scales, lds, rows, M, K, (float*)Y, ldy, s);
  return stream ? dequantize<true>(codes, ldc, scales, lds, rows, M, K, (uint16_t*)Y, ldy, s)
                : dequantize<false>(codes, ldc, scales, lds, rows, M, K, (uint16_t*)Y, ldy, s);
}

hipError_t launch_fp8b_activations(const void* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R,
                                   uint8_t* codes, int64_t ldc, float* scales, int64_t lds, hipStream_t s) {
  return by_rows(R, (K + kFp8Block - 1) / kFp8Block * kLanes, [&](int64_t r0, int64_t n) {
    // rows picked by index keep X's origin
    quantize_rows<true, false>((const uint16_t*)X + (rows ? 0 : r0 * ldx), rows ? M : n, K, ldx,
                               rows ? rows + r0 : nullptr, n, codes + r0 * ldc, ldc, scales + r0 * lds, lds, s);
  });
}

hipError_t launch_fp8b_lay_out(const uint8_t* X, int64_t ldx, const float* sx, int64_t lds_in, int64_t M, int64_t K,
                               const int32_t* rows, int64_t R, uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                               hipStream_t s) {
  return by_rows(R, ldc / 16, [&](int64_t r0, int64_t n) {
    const int64_t x0 = rows ? 0 : r0;
    lay_out_kernel<<<groups_of(n * (ldc / 16)), 256, 0, s>>>(X + x0 * ldx, ldx, sx + x0 * lds_in, lds_in, rows ? M : n, K,
                                                             rows ? rows + r0 : nullptr, n, codes + r0 * ldc, ldc,
                                                             scales + r0 * lds, lds);
  });
}

hipError_t launch_fp8b_pack(const Fp8bDesc& d, const uint8_t* W, int64_t ldw, const float* scales, int64_t lds,
                            hipStream_t s) {
  const hipError_t e = by_rows(d.E * d.NT, d.NU * 128, [&](int64_t t0, int64_t n) {
    pack_kernel<<<groups_of(n * d.NU * 128), 256, 0, s>>>(d, t0, n, W, ldw);
  });
  if (e != hipSuccess) return e;
  return by_rows(d.E * d.SG, d.NUe * 2, [&](int64_t g0, int64_t n) {
    pack_scales_kernel<<<groups_of(n * d.NUe * 2), 256, 0, s>>>(d, g0, n, scales, lds);
  });
}

}  // namespace spense
