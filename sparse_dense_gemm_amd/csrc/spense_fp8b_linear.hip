// HIP kernel of the products with packed block-scaled e4m3 weights (fp8b), for
// one weight matrix or a set of experts whose activation rows are grouped by
// expert in runs of any length.
//
//   Y[r, n] = sum_b sx[r, b] sw[n, b] sum_(k in b) x[r, k] w_e[n, k],   o_e <= r < o_(e+1),
//
// over blocks b of 128 columns: with codes x the inner sum is one 16x16x128
// product, with bf16 x (sx = 1) four 16x16x32 products on the weights widened
// exactly in registers.  It starts from zero and is added to the sums by a fused
// multiply-add with the product of the two scales, in 32 bits: a scale that is no
// power of two cannot go through the matrix instruction's own scale operand, and
// rounding it into an operand would lose bits.  That is four vector instructions
// to each 16x16x128, which takes the time of eight, so they run beside it.
//
// Tiles, launch order, split K and the way into Y are those of the products in
// spense_experts.hip: a workgroup owns NW R row tiles (16 R NW output columns)
// and up to 16 T activation rows of one expert; weights stream from memory into
// each wave's registers through a ring of D stages, activations are copied into
// LDS, D stages at a time into one of two buffers while the other is read.  A
// stage is 256 bytes of every row: 128 bf16 columns or 256 codes.
#include "spense_experts_device.h"
#include "spense_fp8b.h"

namespace spense {
namespace {

// Configurations: X(index, waves, row tiles per wave R, m-tiles T, stages D in
// the ring and in an LDS buffer, waves per SIMD the registers allow)
#define SPENSE_FP8B_CODES_CONFIGS(X) \
  X(0, 8, 1, 1, 8, 2)                \
  X(1, 4, 1, 2, 4, 2)                \
  X(2, 8, 1, 4, 2, 2)                \
  X(3, 4, 2, 8, 1, 2)                \
  X(4, 4, 4, 8, 1, 2)
#define SPENSE_FP8B_BF16_CONFIGS(X) \
  X(0, 8, 1, 1, 8, 2)               \
  X(1, 4, 1, 2, 4, 2)               \
  X(2, 8, 1, 4, 2, 2)               \
  X(3, 4, 2, 8, 1, 2)               \
  X(4, 4, 4, 4, 1, 2)

__device__ __forceinline__ f32x4 mfma_bf16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// the sum of one block of 128 columns, from zero
__device__ __forceinline__ f32x4 mfma_e4m3(const u32x4& a0, const u32x4& a1, const u32x4& b0, const u32x4& b1) {
  const u32x8 A = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
  const u32x8 B = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, A), __builtin_bit_cast(i32x8, B),
                                                          f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// XQ: activations are codes (true) or bf16 (false)
template <bool XQ, int NW, int R, int T, int D, int WPS>
__global__ __launch_bounds__(NW * 64, WPS) void fp8b_kernel(Fp8bDesc d, Fp8bArgs a, ExpertsPlan p) {
  constexpr int kRows = 16 * T;
  constexpr int NU = XQ ? 2 : 1;                         // units of a stage
  constexpr uint32_t kStage = kRows * kStageBytes;       // a stage's rows in LDS
  constexpr uint32_t kScales = XQ ? kRows * 8u : 0u;     // and their scales: [row][unit]
  constexpr uint32_t kBuf = D * (kStage + kScales);
  constexpr int NL = 2 * NU;                             // 16-byte weight loads per row tile and stage
  constexpr int kLoads = R * NL + 1;                     // with the weights' scales: loads per wave and stage
  constexpr int kWait = D * kLoads;                      // and of the whole ring
  static_assert(kWait < 64, "the wait fits the counter");
  // With one stage in the ring its copies are spread over the first products,
  // and its scales are loaded a stage ahead.
  constexpr bool kSpread = D == 1;
  constexpr int kYoung = kSpread ? R * NL : kWait;       // weight loads after the last copy
  __shared__ __attribute__((aligned(1024))) uint8_t xb[2 * kBuf];
  __shared__ int last_flag;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4;

  // ---- which tile ----
  const int S = p.splits;
  int s, rg, j, e, cnt;
  int64_t row0;
  if (!find_tile(d, a, p, kRows, s, rg, j, e, row0, cnt)) return;
  s = __builtin_amdgcn_readfirstlane(s);
  rg = __builtin_amdgcn_readfirstlane(rg);
  j = __builtin_amdgcn_readfirstlane(j);
  e = __builtin_amdgcn_readfirstlane(e);
  cnt = __builtin_amdgcn_readfirstlane(cnt);
  row0 = (int64_t)__builtin_amdgcn_readfirstlane((int)row0);
  const int nst = (int)((d.NU + NU - 1) / NU);  // stages of K
  int lo, hi;
  split_range(nst, s, S, lo, hi);
  const int n = hi - lo;

  // ---- weights: this wave's row tiles (those past the last read zeros), which
  // lie in one group of 128 packed rows ----
  const int64_t rt0 = (int64_t)rg * (NW * R) + wave * R;
  const int64_t nrt = d.NT - rt0 <= 0 ? 0 : d.NT - rt0 < R ? d.NT - rt0 : R;
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(d.wpack + ((int64_t)e * d.NT + (nrt ? rt0 : 0)) * d.tile_bytes, (uint32_t)(nrt * d.tile_bytes));
  static_assert(8 % R == 0, "a wave's row tiles share their scales");
  const __amdgpu_buffer_rsrc_t sr =
      make_rsrc(d.scales + ((int64_t)e * d.SG + (nrt ? rt0 / 8 : 0)) * d.NUe * 2, (uint32_t)(d.NUe * 8));
  const uint32_t tb = (uint32_t)d.tile_bytes;
  u32x4 w[D][R][NL];
  float sw[kSpread ? 2 : D][2 * NU];  // [unit][even, odd packed rows]
  auto load_w = [&](auto slot, int r, int i, int c) __attribute__((always_inline)) {
    const int st = lo + c;
    const bool in = c < n && (!XQ || 2 * st + i / 2 < (int)d.NU);
    w[decltype(slot)::value][r][i] =
        buf_load16(wr, 16 * lane, in ? (uint32_t)r * tb + (uint32_t)(NL * st + i) * 1024u : kOutOfRange);
  };
  auto load_scales = [&](auto slot, int c) __attribute__((always_inline)) {
    const uint32_t off = c < n ? (uint32_t)(lo + c) * (8u * NU) : kOutOfRange;
    float(&o)[2 * NU] = sw[decltype(slot)::value];
    if constexpr (XQ) {
      const f32x4 v = __builtin_bit_cast(f32x4, buf_load16(sr, 0, off));
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = v[i];
    } else {
      const f32x2 v = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, 0, (int)off, 0));
      o[0] = v.x;
      o[1] = v.y;
    }
  };

  // ---- activations.  A copy takes four rows x 256 bytes: lane l row l / 16,
  // piece (l % 16) ^ ((row - 4) % 16) of 16 bytes.  A read of 16 bytes a lane
  // serves 16 lanes at a time, rows 0-3 and 12-15 of one piece with rows 4-11 of
  // the next lane group's: with that shift they hit different banks for both
  // orders of the pieces, which differ between lane groups in the low three bits
  // or agree in the high one.  Rows past the group and bytes past the row take an
  // offset beyond the resource and land as zeros. ----
  constexpr int kQ = 4 * T;                           // copies of a stage
  constexpr int kPer = D * kQ / NW;                   // copies of a buffer per wave
  constexpr int kRowsPer = kQ >= NW ? kQ / NW : 1;    // different rows among them
  static_assert(NW % 4 == 0, "a wave's copies have the same rows modulo 16");
  static_assert(D * kQ % NW == 0 && (kQ % NW == 0 || NW % kQ == 0), "every wave copies the same share");
  const int64_t xrow0 = a.rows ? 0 : row0;
  const int64_t xrows = a.rows ? a.M : cnt;
  const i32x4 xr = rsrc_words(a.X + xrow0 * a.ldx, (uint32_t)((xrows - 1) * a.ldx + a.xbytes));
  auto x_row = [&](int local) -> uint32_t {  // row of X behind row `local` of the group, or out of range
    if (local >= cnt) return 0xFFFFFFFFu;
    if (!a.rows) return (uint32_t)local;
    const int64_t q = a.rows[row0 + local];
    return q < 0 || q >= a.M ? 0xFFFFFFFFu : (uint32_t)q;
  };
  const int q0 = kQ >= NW ? wave : wave % kQ;
  const int cr = lane >> 4, piece = (lane & 15) ^ ((4 * (q0 & 3) + cr - 4) & 15);
  uint32_t xo[kRowsPer];
#pragma unroll
  for (int i = 0; i < kRowsPer; ++i) {
    const uint32_t r = x_row(4 * (q0 + NW * i) + cr);
    xo[i] = r == 0xFFFFFFFFu ? kOutOfRange : r * (uint32_t)a.ldx + 16u * piece;
  }
  // scales of codes: a copy takes 32 (row, unit) pairs twice over, lane l pair l of [stage][row][unit]
  constexpr int kSC = XQ ? D * kRows * 2 / 64 : 0;    // copies of a buffer (D T is even)
  constexpr int kSPer = XQ ? (kSC + NW - 1) / NW : 1;
  static_assert(!XQ || D * kRows * 2 % 64 == 0, "whole copies");
  uint32_t xso[kSPer];
  i32x4 xsr{};
  if constexpr (XQ) {
    xsr = rsrc_words(a.xs + xrow0 * a.ldxs, (uint32_t)((xrows - 1) * a.ldxs + 4 * d.NU));
#pragma unroll
    for (int i = 0; i < kSPer; ++i) {
      const int at = 64 * (wave + NW * i) + lane;
      const uint32_t r = x_row((at >> 1) % kRows);
      xso[i] = r == 0xFFFFFFFFu ? kOutOfRange : r * (uint32_t)a.ldxs + 4u * (at & 1);
    }
  }
  // copy number i (a compile-time index) of this wave's share of stages c ..
  // c + D - 1 of the split: first the rows, then the scales
  constexpr int kCopies = kPer + (XQ ? kSPer : 0);
  auto copy_one = [&](int c, uint32_t buf, auto ic) __attribute__((always_inline)) {
    constexpr int i = decltype(ic)::value;
    if constexpr (i < kPer) {
      const int q = kQ >= NW ? wave + NW * (i % kRowsPer) : q0;
      const int st = kQ >= NW ? i / kRowsPer : wave / kQ + i * (NW / kQ);
      const int at = lo + c + st;  // stage of K
      const int left = (int)a.xbytes - at * kStageBytes;
      const uint32_t v = 16 * piece >= left || at >= hi ? kOutOfRange : xo[i % kRowsPer];
      copy16<false>(xr, buf + st * kStage + q * 1024u, v, (uint32_t)(at < hi ? at * kStageBytes : 0));
    } else {
      const int id = wave + NW * (i - kPer);
      const int st = (64 * id + lane) / (2 * kRows), at = lo + c + st;  // one stage for all lanes, or several
      if (kSC % NW == 0 || id < kSC) {
        const bool in = at < hi && 2 * at + (lane & 1) < (int)d.NU;
        copy4<false>(xsr, buf + D * kStage + id * 256u, in ? xso[i - kPer] + (uint32_t)at * 8u : kOutOfRange, 0u);
      }
    }
  };
  auto copy_x = [&](int c, uint32_t buf) __attribute__((always_inline)) {
    static_for<0, kCopies>([&](auto ic) __attribute__((always_inline)) { copy_one(c, buf, ic); });
  };

  // this lane's pieces of row lane % 16: codes, unit i / 2, half i % 2; bf16, step i
  const int fr = lane & 15;
  uint32_t fo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pc = XQ ? 8 * (i >> 1) + 2 * g + (i & 1) : 4 * g + i;
    fo[i] = (uint32_t)(fr * kStageBytes + 16 * (pc ^ ((fr - 4) & 15)));
  }

  f32x4 acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a block's sum into the sums: s0 for even packed rows, s1 for odd ones
  auto add = [&](f32x4& y, const f32x4& v, float s0, float s1) __attribute__((always_inline)) {
    y[0] = fmaf(v[0], s0, y[0]);
    y[1] = fmaf(v[1], s1, y[1]);
    y[2] = fmaf(v[2], s0, y[2]);
    y[3] = fmaf(v[3], s1, y[3]);
  };

  const uint32_t xlds = lds_addr(xb);
  copy_x(0, xlds);
  // in the loop's order: the compiler's waits count the loads issued since
  static_for<0, D>([&](auto sl) __attribute__((always_inline)) {
    if constexpr (kSpread) load_scales(sl, decltype(sl)::value);
    static_for<0, NL>([&](auto ic) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < R; ++r) load_w(sl, r, decltype(ic)::value, decltype(sl)::value);
    });
    if constexpr (!kSpread) load_scales(sl, decltype(sl)::value);
    __builtin_amdgcn_sched_barrier(0);
  });
  // Waits until this wave's copies have landed (at most `young` weight loads
  // are younger than they are) and its LDS reads are done, then for the others.
  auto ready = [&](auto young) __attribute__((always_inline)) {
    constexpr int v = decltype(young)::value;
    __builtin_amdgcn_s_waitcnt((int)((v & 15) | ((v >> 4) << 14) | (7 << 4) | (0 << 8)));
    barrier_no_fence();
  };
  ready(std::integral_constant<int, kWait>{});

  uint32_t cur = 0;  // the buffer to read
  for (int c0 = 0; c0 < n; c0 += D) {
    const uint32_t other = xlds + (kBuf - cur);
    if constexpr (!kSpread) copy_x(c0 + D, other);
    if constexpr (kSpread) load_scales(std::integral_constant<int, 1>{}, c0 + 1);
    static_for<0, D>([&](auto sl) __attribute__((always_inline)) {
      constexpr int i = decltype(sl)::value;
      const int c = c0 + i;
      const uint8_t* xs = xb + cur + i * kStage;
      // past the last stage the copies write zeros: no branch in the loop
      auto copies = [&](auto kc, auto steps) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value, N = decltype(steps)::value;
        if constexpr (kSpread && k < N)
          static_for<k * kCopies / N, (k + 1) * kCopies / N>(
              [&](auto ic) __attribute__((always_inline)) { copy_one(c0 + D, other, ic); });
      };
      if constexpr (XQ) {
        // 2 T steps of one operand and its R products; operands and their scales
        // are read a step ahead, a product's sum is taken kLag products later
        constexpr int kLag = R > 1 ? 2 : 1, kRing = kLag + 1;
        const uint8_t* xe = xb + cur + D * kStage + i * kScales + fr * 8;
        u32x4 b[2][2];
        float sx[2], s0[2], s1[2];
        f32x4 P[kRing];
        auto read_b = [&](auto kc) __attribute__((always_inline)) {
          constexpr int k = decltype(kc)::value, q = k / T, t = k % T;
          if constexpr (k < 2 * T) {
            b[k & 1][0] = *(const u32x4*)(xs + t * (16 * kStageBytes) + fo[2 * q]);
            b[k & 1][1] = *(const u32x4*)(xs + t * (16 * kStageBytes) + fo[2 * q + 1]);
            sx[k & 1] = *(const float*)(xe + t * 128 + 4 * q);
          }
        };
        auto take = [&](auto mc) __attribute__((always_inline)) {  // product m of the stage
          constexpr int m = decltype(mc)::value, k = m / R;
          if constexpr (m >= 0) add(acc[m % R][k % T], P[m % kRing], s0[k & 1], s1[k & 1]);
        };
        read_b(std::integral_constant<int, 0>{});
        static_for<0, 2 * T>([&](auto kc) __attribute__((always_inline)) {
          constexpr int k = decltype(kc)::value, q = k / T, t = k % T;
          read_b(std::integral_constant<int, k + 1>{});
          s0[k & 1] = sx[k & 1] * sw[i][2 * q];
          s1[k & 1] = sx[k & 1] * sw[i][2 * q + 1];
          static_for<0, R>([&](auto rc) __attribute__((always_inline)) {
            constexpr int r = decltype(rc)::value, m = k * R + r;
            P[m % kRing] = mfma_e4m3(w[i][r][2 * q], w[i][r][2 * q + 1], b[k & 1][0], b[k & 1][1]);
            take(std::integral_constant<int, m - kLag>{});
          });
          copies(kc, std::integral_constant<int, (T >= 2 ? T / 2 : 1)>{});
          if constexpr (t == T - 1) {  // refill what this unit was the last to read
            static_for<0, 2>([&](auto hc) __attribute__((always_inline)) {
#pragma unroll
              for (int r = 0; r < R; ++r) load_w(sl, r, 2 * q + decltype(hc)::value, c + D);
            });
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        static_for<2 * T * R - kLag, 2 * T * R>(take);
        if constexpr (!kSpread) load_scales(sl, c + D);
      } else {
        // T steps of four operands and their 4 R products, whose sums are taken
        // in the next step; the unit's weights are widened first, so that their
        // registers are free for the loads of stage c + D
        bf16x8 A[4][R];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const u32x4& v = w[i][r][q >> 1];
            A[q][r] = q & 1 ? fp8x8_to_bf16(v.z, v.w) : fp8x8_to_bf16(v.x, v.y);
          }
        u32x4 b[2][4];
        f32x4 P[R];
        auto read_b = [&](auto tc) __attribute__((always_inline)) {
          constexpr int t = decltype(tc)::value;
          if constexpr (t < T)
#pragma unroll
            for (int q = 0; q < 4; ++q) b[t & 1][q] = *(const u32x4*)(xs + t * (16 * kStageBytes) + fo[q]);
        };
        read_b(std::integral_constant<int, 0>{});
        constexpr int kFirst = T >= 4 ? T / 4 : 1;  // steps that the copies are spread over
        static_for<0, T>([&](auto tc) __attribute__((always_inline)) {
          constexpr int t = decltype(tc)::value;
          read_b(std::integral_constant<int, t + 1>{});
          static_for<0, 4>([&](auto qc) __attribute__((always_inline)) {
            constexpr int q = decltype(qc)::value;
#pragma unroll
            for (int r = 0; r < R; ++r) {
              if constexpr (q == 0 && t > 0) add(acc[r][t - 1], P[r], sw[i][0], sw[i][1]);
              P[r] = mfma_bf16(A[q][r], as_bf16x8(b[t & 1][q]), q == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : P[r]);
            }
          });
          copies(tc, std::integral_constant<int, kFirst>{});
          if constexpr (t == kFirst - 1) {
            static_for<0, NL>([&](auto hc) __attribute__((always_inline)) {
#pragma unroll
              for (int r = 0; r < R; ++r) load_w(sl, r, decltype(hc)::value, c + D);
            });
          }
          __builtin_amdgcn_sched_barrier(0);
        });
#pragma unroll
        for (int r = 0; r < R; ++r) add(acc[r][T - 1], P[r], sw[i][0], sw[i][1]);
        if constexpr (!kSpread) load_scales(sl, c + D);
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    // the other buffer has landed and this one's reads are done
    ready(std::integral_constant<int, kYoung>{});
    if constexpr (kSpread) {
#pragma unroll
      for (int k = 0; k < 2 * NU; ++k) sw[0][k] = sw[1][k];
    }
    cur = kBuf - cur;
  }
  SPENSE_WAIT_VM(0);

  static_assert(NW * kPartLds<R> <= 2 * kBuf, "the waves' parts of LDS");
  finish<R, T>(d, a, p, acc, xb + wave * kPartLds<R>, s, rg, j, rt0, row0, cnt, &last_flag);
}

template <bool XQ, int NW, int R, int T, int D, int WPS>
hipError_t launch_k(const Fp8bDesc& d, const Fp8bArgs& a, const ExpertsPlan& p, hipStream_t s) {
  const unsigned grid = grid_of(d, p, NW * R, NW * 64);
  if (!grid) return hipErrorInvalidValue;
  fp8b_kernel<XQ, NW, R, T, D, WPS><<<grid, NW * 64, 0, s>>>(d, a, p);
  return hipGetLastError();
}

}  // namespace

int fp8b_config_count(bool codes) {
  int n = 0;
#define SPENSE_FP8B_COUNT(i, nw, r, t, dd, wps) ++n;
  if (codes) {
    SPENSE_FP8B_CODES_CONFIGS(SPENSE_FP8B_COUNT)
  } else {
    SPENSE_FP8B_BF16_CONFIGS(SPENSE_FP8B_COUNT)
  }
#undef SPENSE_FP8B_COUNT
  return n;
}

ExpertsShape fp8b_shape(bool codes, int config) {
#define SPENSE_FP8B_SHAPE(i, nw, r, t, dd, wps) \
  if (config == i) return ExpertsShape{nw, r, t, dd};
  if (codes) {
    SPENSE_FP8B_CODES_CONFIGS(SPENSE_FP8B_SHAPE)
  } else {
    SPENSE_FP8B_BF16_CONFIGS(SPENSE_FP8B_SHAPE)
  }
#undef SPENSE_FP8B_SHAPE
  return ExpertsShape{0, 0, 0, 0};
}

hipError_t launch_fp8b_linear(const Fp8bDesc& d, const Fp8bArgs& a, const ExpertsPlan& p, hipStream_t s) {
#define SPENSE_FP8B_CASE(xq, i, nw, r, t, dd, wps) \
  case i: return launch_k<xq, nw, r, t, dd, wps>(d, a, p, s);
  if (a.codes) {
    switch (p.config) {
#define SPENSE_FP8B_CODES_CASE(...) SPENSE_FP8B_CASE(true, __VA_ARGS__)
      SPENSE_FP8B_CODES_CONFIGS(SPENSE_FP8B_CODES_CASE)
#undef SPENSE_FP8B_CODES_CASE
    }
  } else {
    switch (p.config) {
#define SPENSE_FP8B_BF16_CASE(...) SPENSE_FP8B_CASE(false, __VA_ARGS__)
      SPENSE_FP8B_BF16_CONFIGS(SPENSE_FP8B_BF16_CASE)
#undef SPENSE_FP8B_BF16_CASE
    }
  }
#undef SPENSE_FP8B_CASE
  return hipErrorInvalidValue;
}

}  // namespace spense
