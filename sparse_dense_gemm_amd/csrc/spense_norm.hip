// HIP kernels of the pass over the rows between two blocks of a decoder:
//
//   o = O[t], or sum_j weights[t, j] O[pos[t, j]]
//   r = scale * residual + gate * (post ? o / sqrt(mean(o^2) + eps) * post : o)
//   y = r / sqrt(mean(r^2) + eps) * pre
//
// r goes out rounded once, y (from the unrounded r) as fp32, bf16 or e4m3 codes
// with a scale for each block of 128 columns.
//
// One launch reads and writes every operand once: a workgroup takes a row, which
// stays in registers between the two sums (a wave a row would hold 80 values a lane
// at 5120 columns, and few rows would leave the chip empty).  Bound by memory: 8191
// rows of 5120 (bf16 in, residual and gate in fp32 and bf16, codes out) 99 us, 464 MB
// at 4.7 TB/s; 2048 rows of 5120, each the sum of two fp32 rows, 28 us, 147 MB at 5.3.
// Above 6144 columns a CU holds one workgroup, whose loads, barriers and stores
// nothing covers: 7168, 8192 and 27648 columns 107, 104 and 110 us for the same bytes,
// and the sums of 8192 and 12288 columns 30 and 40 (four pieces a thread, of which the
// sums of fp32 rows spill 36 to 116 bytes a lane; so does an fp32 residual with bf16
// rows of a length that is no multiple of eight, 36 bytes).
// One row takes 3.0 us, most of it the launch and the wait for its loads.
#include <algorithm>
#include <cfloat>

#include "spense_fp8b_device.h"

namespace spense {
namespace {

constexpr int kMaxThreads = 1024;

// Sum over the lanes of a row of sixteen, then over the wave, in every lane.
__device__ __forceinline__ float row_sum(float v) {
  auto add = [&](int o) { v += __int_as_float(o); };
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x122, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x121, 0xF, 0xF, false));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0)) +
         __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16)) +
         __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32)) +
         __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
}

// Sum over the workgroup (at most sixteen waves), in a fixed order.  tmp: 16
// floats of LDS that no other sum in flight uses.
__device__ __forceinline__ float block_sum(float v, float* tmp) {
  v = wave_sum(v);
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  const int i = threadIdx.x & 15;
  return row_sum(i < waves ? tmp[i] : 0.f);
}

// 1 / sqrt(s / H + eps), rh = 1 / H.  Every finite sum is divided; an infinite one
// gives 0, as in the formula, and a NaN a NaN.  The root instruction is off by up to
// a unit in the last place, which one step takes to little more than half of one
// (t + d is x r exactly); eps is a normal number, so x is.  It costs ten
// instructions a row.  A block of codes does not see the second norm's factor, up to
// roundings: its scale takes that up.
__device__ __forceinline__ float rms_scale(float s, const spense_norm& n, float rh) {
  const float x = (s <= FLT_MAX ? quotient(s, (float)n.H, rh) : s) + n.eps;
  const float r = __builtin_amdgcn_rsqf(x);
  const float t = x * r, d = fmaf(x, r, -t);
  const float e = fmaf(-d, r, fmaf(-t, r, 1.0f));
  const float better = fmaf(0.5f * r, e, r);
  return r > 0.f ? better : r;  // x infinite
}

// The end of a row of H columns.  kWhole: H is a multiple of eight.  kShift: at
// least eight; the last piece of a row is its last eight columns, of which it
// leaves out the d that the piece before has (in place those may be stored already
// when it reads them), so that no lane branches around its loads: 6731 rows of 574
// columns, each of four fp32 rows, 18.5 us, 29.5 with the last lane's values loaded
// one by one.  kAny: one by one.
enum Ends { kWhole, kShift, kAny };

// Eight values of a row as they are stored: loads go out together and are widened
// where they are used (a widening beside its load is a wait for it).
template <typename XT>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 a;
  template <Ends E>
  __device__ __forceinline__ void load(const uint16_t* x, int64_t k, int64_t H) {
    if constexpr (E == kShift) k = k + 8 <= H ? k : H - 8;
    if (E != kAny || k + 8 <= H) {
      a = *(const u32x4_any*)(x + k);
    } else {
      a = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < H) a[i >> 1] |= (uint32_t)x[k + i] << (16 * (i & 1));
    }
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? a[i >> 1] & 0xFFFF0000u : a[i >> 1] << 16);
  }
};
template <>
struct Raw<float> {
  f32x4 a, b;
  template <Ends E>
  __device__ __forceinline__ void load(const float* x, int64_t k, int64_t H) {
    if constexpr (E == kShift) k = k + 8 <= H ? k : H - 8;
    if (E != kAny || k + 8 <= H) {
      a = *(const f32x4_any*)(x + k);
      b = *(const f32x4_any*)(x + k + 4);
    } else {
      a = b = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (k + i < H) (i < 4 ? a : b)[i & 3] = x[k + i];
    }
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i] : b[i - 4]; }
};
// the same of a type known at the call
struct RawAny {
  Raw<float> f;
  Raw<uint16_t> h;
  template <Ends E>
  __device__ __forceinline__ void load(const void* p, bool f32, int64_t row, int64_t k, int64_t H) {
    if (f32) f.load<E>((const float*)p + row, k, H);
    else h.load<E>((const uint16_t*)p + row, k, H);
  }
  __device__ __forceinline__ void multiply(bool f32, float (&v)[8]) const {
    if (f32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= f.get(i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= h.get(i);
    }
  }
};

// Columns k .. k + 7 of a row's operands (kShift: at the row's end H - 8 .. H - 1).
// OT, RT: types of O and of the residual; POS: O's rows are summed over j.  Columns
// from H on are zeros.
template <typename OT, typename RT, bool POS, Ends E>
struct Piece {
  Raw<OT> o[POS ? 2 : 1];
  Raw<RT> res;
  RawAny gate, post, pre;
  float w[2];

  __device__ __forceinline__ void load_row(const spense_norm& n, int64_t t, int64_t k) {
    if constexpr (POS) load_two(n, t, k, 0);
    else o[0].template load<E>((const OT*)n.O + t * n.ldo, k, n.H);
    if (n.residual) res.template load<E>((const RT*)n.residual + t * n.ldr, k, n.H);
  }
  // rows j0 and j0 + 1 of the sum over j
  __device__ __forceinline__ void load_two(const spense_norm& n, int64_t t, int64_t k, int j0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      w[j] = 0.f;
      if (j0 + j >= n.k) continue;
      const int64_t at = n.pos[t * n.k + j0 + j];
      if (at < 0 || at >= n.O_rows) continue;
      w[j] = n.weights[t * n.k + j0 + j];
      o[j].template load<E>((const OT*)n.O + at * n.ldo, k, n.H);
    }
  }
  __device__ __forceinline__ void load_gate(const spense_norm& n, int64_t t, int64_t k) {
    if (n.post) post.load<E>(n.post, n.wtype == DT_F32, 0, k, n.H);
    if (n.gate) gate.load<E>(n.gate, n.gtype == DT_F32, t * n.ldg, k, n.H);
  }
  __device__ __forceinline__ void load_pre(const spense_norm& n, int64_t k) {
    if (n.Y && n.pre) pre.load<E>(n.pre, n.wtype == DT_F32, 0, k, n.H);
  }

  __device__ __forceinline__ void get_o(const spense_norm& n, int64_t t, int64_t k, float (&v)[8]) {
    if constexpr (!POS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = o[0].get(i);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      for (int j0 = 0;;) {  // in the order of j
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int64_t at = j0 + j < n.k ? n.pos[t * n.k + j0 + j] : -1;
          if (at < 0 || at >= n.O_rows) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf(w[j], o[j].get(i), v[i]);
        }
        j0 += 2;
        if (j0 >= n.k) break;
        load_two(n, t, k, j0);
      }
    }
  }
  // r from o times `inv` (1 without a norm after the block)
  __device__ __forceinline__ void get_r(const spense_norm& n, float inv, float (&v)[8]) const {
    if (n.post) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= inv;
      post.multiply(n.wtype == DT_F32, v);
    }
    if (n.gate) gate.multiply(n.gtype == DT_F32, v);
    if (n.residual) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(n.scale, res.get(i), v[i]);
    }
  }
  __device__ __forceinline__ void get_y(const spense_norm& n, float inv, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    if (n.pre) pre.multiply(n.wtype == DT_F32, v);
  }
};

// Values that the piece before has, left out of sums and of a block's maximum.
template <Ends E>
__device__ __forceinline__ void drop(float (&v)[8], int d) {
  if (E == kShift && d > 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i) v[i] = i < d ? 0.f : v[i];
  }
}

template <Ends E, bool STREAM, typename YT>
__device__ __forceinline__ void put8(const spense_norm& n, YT* y, int64_t k, int d, const float (&v)[8]) {
  if (E == kShift && d > 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i >= d) {
        if constexpr (sizeof(YT) == 2) y[k - d + i] = (YT)bf16_rne(v[i]);
        else y[k - d + i] = v[i];
      }
  } else {
    store_row8<STREAM>(y, k, E == kAny ? n.H : k + 8, v);
  }
}

// y out, of all sixteen lanes that share a block (in: columns below H)
template <Ends E, bool STREAM>
__device__ __forceinline__ void put_y(const spense_norm& n, int64_t t, int64_t k, int d, bool in, const float (&y)[8]) {
  if (n.ytype == DT_FP8) {
    const float s = block_scale(row_max(in ? top8(y) : 0u));
    if (!in) return;
    uint8_t* out = (uint8_t*)n.Y + t * n.ldy;
    const u32x2 c = codes8(y, s);
    if (E == kShift && d > 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i >= d) out[k - d + i] = (uint8_t)(c[i >> 2] >> (8 * (i & 3)));
    } else {
      store_codes8<STREAM>(out, k, E == kAny ? n.H : k + 8, c);
    }
    if (k % kFp8Block == 0) n.yscales[t * n.lds + k / kFp8Block] = s;
  } else if (in) {
    if (n.ytype == DT_F32) put8<E, STREAM>(n, (float*)n.Y + t * n.ldy, k, d, y);
    else put8<E, STREAM>(n, (uint16_t*)n.Y + t * n.ldy, k, d, y);
  }
}

__device__ __forceinline__ float sum_of_squares(const float (&v)[8]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
  return s;
}

// A workgroup takes a row, a thread C pieces of eight columns, in registers
// between the sums.  Eight columns are one load of bf16.
template <typename OT, typename RT, bool POS, Ends E, bool STREAM, int C>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(spense_norm n, float rh) {
  __shared__ float tmp[2][16];
  const int64_t t = blockIdx.x;
  const int64_t step = (int64_t)blockDim.x * 8, k0 = (int64_t)threadIdx.x * 8;
  // several pieces: no registers for the weights and gates, which are loaded where they are used
  constexpr bool kHold = C == 1;
  Piece<OT, RT, POS, E> p[C];
  float v[C][8];
  bool in[C];
  int d[C];  // columns at the piece's beginning that the one before has
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k = k0 + c * step;
    in[c] = k < n.H;
    d[c] = E == kShift && in[c] && k + 8 > n.H ? (int)(k + 8 - n.H) : 0;
    if (in[c]) p[c].load_row(n, t, k);
  }
  if constexpr (kHold) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c]) {
        p[c].load_gate(n, t, k0 + c * step);
        p[c].load_pre(n, k0 + c * step);
      }
  }
  float inv = 1.f, s = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (in[c]) p[c].get_o(n, t, k0 + c * step, v[c]);
  if (n.post) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (in[c]) {
        drop<E>(v[c], d[c]);
        s += sum_of_squares(v[c]);
      }
    inv = rms_scale(block_sum(s, tmp[0]), n, rh);
    s = 0.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
    if (in[c]) {
      const int64_t k = k0 + c * step;
      if constexpr (!kHold) p[c].load_gate(n, t, k);
      p[c].get_r(n, inv, v[c]);
      if (n.residual_out) put8<E, STREAM>(n, (RT*)n.residual_out + t * n.ldro, k, d[c], v[c]);
      drop<E>(v[c], d[c]);
      s += sum_of_squares(v[c]);
    }
  if (!n.Y) return;
  inv = rms_scale(block_sum(s, tmp[1]), n, rh);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t k = k0 + c * step;
    if (in[c]) {
      if constexpr (!kHold) p[c].load_pre(n, k);
      p[c].get_y(n, inv, v[c]);
      drop<E>(v[c], d[c]);
    }
    put_y<E, STREAM>(n, t, k, d[c], in[c], v[c]);
  }
}

// Rows that do not fit the registers of a workgroup, read again for each sum, and
// rows of fewer than eight columns.
template <typename OT, typename RT, bool POS, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void norm_long_kernel(spense_norm n, float rh) {
  __shared__ float tmp[2][16];
  const int64_t t = blockIdx.x;
  const int64_t step = (int64_t)blockDim.x * 8, k0 = (int64_t)threadIdx.x * 8;
  float inv = 1.f, inv2 = 1.f, s = 0.f;
  Piece<OT, RT, POS, kAny> p;
  float v[8];
  auto get_r = [&](int64_t k) __attribute__((always_inline)) {
    p.load_row(n, t, k);
    p.load_gate(n, t, k);
    p.get_o(n, t, k, v);
    p.get_r(n, inv, v);
  };
  if (n.post) {
    for (int64_t k = k0; k < n.H; k += step) {
      p.load_row(n, t, k);
      p.get_o(n, t, k, v);
      s += sum_of_squares(v);
    }
    inv = rms_scale(block_sum(s, tmp[0]), n, rh);
    s = 0.f;
  }
  if (n.Y) {
    for (int64_t k = k0; k < n.H; k += step) {
      get_r(k);
      s += sum_of_squares(v);
    }
    inv2 = rms_scale(block_sum(s, tmp[1]), n, rh);
  }
  // every lane takes part in a block's maximum; a thread writes what it alone has
  // read (residual_out may be residual)
  for (int64_t kb = 0; kb < n.H; kb += step) {
    const int64_t k = kb + k0;
    const bool in = k < n.H;
    if (in) {
      get_r(k);
      if (n.residual_out) put8<kAny, STREAM>(n, (RT*)n.residual_out + t * n.ldro, k, 0, v);
    }
    if (!n.Y) continue;
    if (in) {
      p.load_pre(n, k);
      p.get_y(n, inv2, v);
    }
    put_y<kAny, STREAM>(n, t, k, 0, in, v);
  }
}

template <typename OT, typename RT, bool POS, bool STREAM>
hipError_t launch(const spense_norm& n, hipStream_t s) {
  const unsigned T = (unsigned)n.T;
  const int64_t pieces = (n.H + 7) / 8;
  const bool whole = n.H % 8 == 0;
  const float rh = 1.0f / (float)n.H;
  auto threads = [&](int64_t c) { return (unsigned)(((pieces + c - 1) / c + 63) / 64 * 64); };
  if (n.H < 8) {
    norm_long_kernel<OT, RT, POS, STREAM><<<T, 64, 0, s>>>(n, rh);
  } else if (pieces <= kMaxThreads) {
    auto k = whole ? norm_kernel<OT, RT, POS, kWhole, STREAM, 1> : norm_kernel<OT, RT, POS, kShift, STREAM, 1>;
    k<<<T, threads(1), 0, s>>>(n, rh);
  } else if (pieces <= 4 * kMaxThreads) {
    auto k = whole ? norm_kernel<OT, RT, POS, kWhole, STREAM, 4> : norm_kernel<OT, RT, POS, kShift, STREAM, 4>;
    k<<<T, threads(4), 0, s>>>(n, rh);
  } else {
    norm_long_kernel<OT, RT, POS, STREAM><<<T, kMaxThreads, 0, s>>>(n, rh);
  }
  return hipGetLastError();
}

template <typename OT, typename RT>
hipError_t launch_types(const spense_norm& n, bool stream, hipStream_t s) {
  if (n.pos) return stream ? launch<OT, RT, true, true>(n, s) : launch<OT, RT, true, false>(n, s);
  return stream ? launch<OT, RT, false, true>(n, s) : launch<OT, RT, false, false>(n, s);
}

}  // namespace

hipError_t launch_block_norm(const spense_norm& n, hipStream_t s) {
  // a launch's grid counts threads in 32 bits
  constexpr int64_t kMost = (int64_t(1) << 30) / kMaxThreads;
  auto bytes = [](int32_t t) { return t == DT_F32 ? 4 : t == DT_BF16 ? 2 : 1; };
  const int64_t per = (n.residual_out ? bytes(n.rtype) : 0) + (n.Y ? bytes(n.ytype) : 0);
  const bool stream = n.T * n.H * per > kStreamBytes, r32 = n.rtype == DT_F32;
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
    const hipError_t e =
        n.otype == DT_F32
            ? (r32 ? launch_types<float, float>(m, stream, s) : launch_types<float, uint16_t>(m, stream, s))
            : (r32 ? launch_types<uint16_t, float>(m, stream, s) : launch_types<uint16_t, uint16_t>(m, stream, s));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace spense
