// HIP kernels of the pass over the rows between two blocks of a decoder:
//
//   o = O[t], or sum_j weights[t, j] O[pos[t, j]]
//   r = scale * residual + gate * (post ? o / sqrt(mean(o^2) + eps) * post : o)
//   y = r / sqrt(mean(r^2) + eps) * pre
//
// r goes out rounded once, y (from the unrounded r) as fp32, bf16 or e4m3 codes
// with a scale for each block of 128 columns.
#include <algorithm>

#include "spense_fp8b_device.h"

namespace spense {
namespace {

constexpr int kMaxThreads = 1024;

// Sum over the workgroup, in a fixed order: over the lanes of a wave, then over
// the waves.  tmp: 16 floats of LDS that no other sum in flight uses.
__device__ __forceinline__ float block_sum(float v, float* tmp) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += tmp[i];
  return s;
}

__device__ __forceinline__ void load_any(const void* p, bool f32, int64_t row, int64_t k, int64_t H, float (&v)[8]) {
  if (f32) load_row8<float>((const float*)p + row, k, H, v);
  else load_row8<uint16_t>((const uint16_t*)p + row, k, H, v);
}

// o[k .. k + 7] of row t
template <typename OT>
__device__ __forceinline__ void load_o(const spense_norm& n, int64_t t, int64_t k, float (&o)[8]) {
  if (!n.pos) {
    load_row8<OT>((const OT*)n.O + t * n.ldo, k, n.H, o);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int64_t j = 0; j < n.k; ++j) {
    const int64_t at = n.pos[t * n.k + j];
    if (at < 0 || at >= n.O_rows) continue;
    const float w = n.weights[t * n.k + j];
    float v[8];
    load_row8<OT>((const OT*)n.O + at * n.ldo, k, n.H, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(w, v[i], o[i]);
  }
}

// r[k .. k + 7] of row t from the block's output times `inv` (1 without a norm after it)
template <typename RT>
__device__ __forceinline__ void sum_r(const spense_norm& n, int64_t t, int64_t k, float inv, const float (&post)[8],
                                      const float (&res)[8], const float (&gate)[8], float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float b = o[i];
    if (n.post) b = b * inv * post[i];
    if (n.gate) b *= gate[i];
    o[i] = n.residual ? fmaf(n.scale, res[i], b) : b;
  }
}

__device__ __forceinline__ void put_y(const spense_norm& n, int64_t t, int64_t k, const float (&y)[8]) {
  if (n.ytype == DT_FP8) {
    const float s = block_scale(row_max(top8(y)));  // sixteen threads to a block
    if (k >= n.H) return;
    store_codes8((uint8_t*)n.Y + t * n.ldy, k, n.H, codes8(y, s));
    if (k % kFp8Block == 0) n.yscales[t * n.lds + k / kFp8Block] = s;
  } else if (n.ytype == DT_F32) {
    store_row8<float>((float*)n.Y + t * n.ldy, k, n.H, y);
  } else {
    store_row8<uint16_t>((uint16_t*)n.Y + t * n.ldy, k, n.H, y);
  }
}

__device__ __forceinline__ float sum_of_squares(const float (&v)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
  return s;
}

// A workgroup takes a row, a thread C pieces of eight columns, in registers
// between the sums.  With up to two pieces the weights' and gates' loads go out
// with the row's; with four there are no registers for them, and they are loaded
// where they are used.
template <typename OT, typename RT, int C>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(spense_norm n) {
  __shared__ float tmp[2][16];
  const int64_t t = blockIdx.x;
  const int64_t step = (int64_t)blockDim.x * 8, k0 = (int64_t)threadIdx.x * 8;
  constexpr bool kHold = C <= 2;
  constexpr int CW = kHold ? C : 1;
  float o[C][8], res[C][8], gate[CW][8], post[CW][8], pre[CW][8];
  auto load_gate = [&](int64_t k, int c) __attribute__((always_inline)) {
    if (n.gate) load_any(n.gate, n.gtype == DT_F32, t * n.ldg, k, n.H, gate[c]);
    if (n.post) load_any(n.post, n.wtype == DT_F32, 0, k, n.H, post[c]);
  };
  auto load_pre = [&](int64_t k, int c) __attribute__((always_inline)) {
    if (n.Y && n.pre) load_any(n.pre, n.wtype == DT_F32, 0, k, n.H, pre[c]);
  };
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k = k0 + c * step;
    load_o<OT>(n, t, k, o[c]);
    if (n.residual) load_row8<RT>((const RT*)n.residual + t * n.ldr, k, n.H, res[c]);
    if constexpr (kHold) {
      load_gate(k, c);
      load_pre(k, c);
    }
  }
  float inv = 1.f;
  if (n.post) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s += sum_of_squares(o[c]);
    inv = 1.f / sqrtf(block_sum(s, tmp[0]) / (float)n.H + n.eps);
  }
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k = k0 + c * step;
    const int w = kHold ? c : 0;
    if constexpr (!kHold) load_gate(k, 0);
    sum_r<RT>(n, t, k, inv, post[w], res[c], gate[w], o[c]);
    if (n.residual_out) store_row8<RT>((RT*)n.residual_out + t * n.ldro, k, n.H, o[c]);
    s += sum_of_squares(o[c]);
  }
  if (!n.Y) return;
  inv = 1.f / sqrtf(block_sum(s, tmp[1]) / (float)n.H + n.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int w = kHold ? c : 0;
    if constexpr (!kHold) load_pre(k0 + c * step, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[c][i] = n.pre ? o[c][i] * inv * pre[w][i] : o[c][i] * inv;
    put_y(n, t, k0 + c * step, o[c]);
  }
}

// Rows that do not fit the registers of a workgroup: read again for each sum.
template <typename OT, typename RT>
__global__ __launch_bounds__(kMaxThreads) void norm_long_kernel(spense_norm n) {
  __shared__ float tmp[2][16];
  const int64_t t = blockIdx.x;
  const int64_t step = (int64_t)blockDim.x * 8, k0 = (int64_t)threadIdx.x * 8;
  float inv = 1.f;
  if (n.post) {
    float s = 0.f;
    for (int64_t k = k0; k < n.H; k += step) {
      float o[8];
      load_o<OT>(n, t, k, o);
      s += sum_of_squares(o);
    }
    inv = 1.f / sqrtf(block_sum(s, tmp[0]) / (float)n.H + n.eps);
  }
  auto r_of = [&](int64_t k, float(&o)[8]) {
    float res[8], gate[8], post[8];
    load_o<OT>(n, t, k, o);
    if (n.residual) load_row8<RT>((const RT*)n.residual + t * n.ldr, k, n.H, res);
    if (n.gate) load_any(n.gate, n.gtype == DT_F32, t * n.ldg, k, n.H, gate);
    if (n.post) load_any(n.post, n.wtype == DT_F32, 0, k, n.H, post);
    sum_r<RT>(n, t, k, inv, post, res, gate, o);
  };
  float inv2 = 1.f;
  if (n.Y) {
    float s = 0.f;
    for (int64_t k = k0; k < n.H; k += step) {
      float o[8];
      r_of(k, o);
      s += sum_of_squares(o);
    }
    inv2 = 1.f / sqrtf(block_sum(s, tmp[1]) / (float)n.H + n.eps);
  }
  // every thread of a row of sixteen lanes takes part in a block's maximum; a
  // thread writes what it alone has read (residual_out may be residual)
  for (int64_t kb = 0; kb < n.H; kb += step) {
    const int64_t k = kb + k0;
    float o[8];
    r_of(k, o);
    if (n.residual_out) store_row8<RT>((RT*)n.residual_out + t * n.ldro, k, n.H, o);
    if (!n.Y) continue;
    float pre[8];
    if (n.pre) load_any(n.pre, n.wtype == DT_F32, 0, k, n.H, pre);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = n.pre ? o[i] * inv2 * pre[i] : o[i] * inv2;
    put_y(n, t, k, o);
  }
}

template <typename OT, typename RT>
hipError_t launch(const spense_norm& n, hipStream_t s) {
  const unsigned T = (unsigned)n.T;
  const int64_t pieces = (n.H + 7) / 8;
  auto threads = [&](int64_t c) { return (unsigned)(((pieces + c - 1) / c + 63) / 64 * 64); };
  if (pieces <= kMaxThreads) norm_kernel<OT, RT, 1><<<T, threads(1), 0, s>>>(n);
  else if (pieces <= 2 * kMaxThreads) norm_kernel<OT, RT, 2><<<T, threads(2), 0, s>>>(n);
  else if (pieces <= 4 * kMaxThreads) norm_kernel<OT, RT, 4><<<T, threads(4), 0, s>>>(n);
  else norm_long_kernel<OT, RT><<<T, kMaxThreads, 0, s>>>(n);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const spense_norm& n, hipStream_t s) {
  // a launch's grid counts threads in 32 bits
  constexpr int64_t kMost = (int64_t(1) << 30) / kMaxThreads;
  auto bytes = [](int32_t t) { return t == DT_F32 ? 4 : t == DT_BF16 ? 2 : 1; };
  for (int64_t t0 = 0; t0 < n.T; t0 += kMost) {
    spense_norm m = n;
    m.T = std::min(n.T - t0, kMost);
    if (n.pos) {
      m.pos += t0 * n.k;
      m.weights += t0 * n.k;
    } else {
      m.O = (const uint8_t*)n.O + t0 * n.ldo * bytes(n.otype);
    }
    if (n.gate) m.gate = (const uint8_t*)n.gate + t0 * n.ldg * bytes(n.gtype);
    if (n.residual) m.residual = (const uint8_t*)n.residual + t0 * n.ldr * bytes(n.rtype);
    if (n.residual_out) m.residual_out = (uint8_t*)n.residual_out + t0 * n.ldro * bytes(n.rtype);
    if (n.Y) m.Y = (uint8_t*)n.Y + t0 * n.ldy * bytes(n.ytype);
    if (n.yscales) m.yscales += t0 * n.lds;
    hipError_t e;
    if (n.otype == DT_F32) e = n.rtype == DT_F32 ? launch<float, float>(m, s) : launch<float, uint16_t>(m, s);
    else e = n.rtype == DT_F32 ? launch<uint16_t, float>(m, s) : launch<uint16_t, uint16_t>(m, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace spense
