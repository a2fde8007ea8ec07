// HIP kernel of the products with packed mx4 or bf16 weights, for one weight
// matrix (the mx4 linear layer) or a set of experts whose activation rows are
// grouped by expert in runs of any length.
//
//   Y[r, n] = sum_k x[r, k] w_e[n, k],   o_e <= r < o_(e+1),
//
// with w (and x, if quantised) = code * 2^(exponent) in blocks of 32 columns.
// Products of two mx4 blocks run on the scaled matrix instruction 16x16x128,
// which takes the codes and the exponent bytes as they are stored; with bf16
// activations mx4 weights are widened exactly in registers and, like bf16
// weights, run on 16x16x32.  Sums are held in 32 bits.
//
// A workgroup owns NW R row tiles (16 R NW output columns) and up to 16 T
// activation rows of one expert.  Weights are read once per workgroup, each
// wave streaming its own row tiles from memory through a ring of D stages in
// registers (they are packed as the matrix instructions' operands, so they
// need neither LDS nor a shuffle); activations are shared by the waves, so
// they are copied into LDS, D stages at a time into one of two buffers while
// the other is read.  A stage is 256 bytes of every row: 128 bf16 columns or
// 512 mx4 columns, in both cases four operands of 16 bytes per lane.
#include "spense_experts_device.h"

namespace spense {
namespace {

// Per pair of operands a wave reads 16 bytes a lane of activations from LDS for
// R products; per stage a workgroup takes R NW weight tiles and 16 T rows through
// the CU's vector cache.  So large groups take the largest block whose sums fit
// the registers of two workgroups per CU, 256 columns x 128 rows (R = 4, T = 8:
// 128 registers): one workgroup's start, barriers and stores are then covered
// by the other's products.  One workgroup of 256 x 256 halves the weights' bytes
// and lost (55296 x 5120, 2048 rows, mx4 x mx4: 307 us, four waves of T = 16
// 489, eight waves with both operands in LDS 324).  128 columns (R = 2) serve
// where that leaves too few blocks.  Below 64 rows the weights' stream from
// memory is all: more waves and a deeper ring, D stages of R row tiles in
// flight per wave (25600 x 5120, one row: 13.2 us, 5.3 TB/s; 5120 x 25600, 32
// rows: 20 us, 3.6 TB/s, its sums split six ways).
//
// What bounds the large ones (12288 x 5120 mx4 with bf16 rows 174-182 us, 1.45
// PFLOP/s; 55296 x 5120 mx4 x mx4 297-309, 3.8; 16 experts of 3200 x 5120
// bf16, 8192 rows, 268-280, 0.97 without padding): the matrix instructions are
// busy in 67, 51 and 58% of the cycles, at a clock that the load brings down to
// 1.6-2.0 GHz; the rest waits for operands (17, 29 and 26 bytes per cycle and CU
// come from L2) and, in the second, for the stores.
//
// The compiler's waits for the weights count loads in order of issue, so loads
// that were issued in another order before the loop, or only on some paths in it,
// make it wait for the youngest: the first loads are in the loop's order, and
// a pass has no branches (stages past the end load zeros).
//
// Configurations: X(index, waves, row tiles per wave R, m-tiles T, stages D in
// the ring and in an LDS buffer, waves per SIMD the registers allow)
#define SPENSE_EXPERT_CONFIGS(X) \
  X(0, 8, 1, 1, 8, 2)            \
  X(1, 4, 1, 2, 4, 2)            \
  X(2, 8, 1, 4, 2, 2)            \
  X(3, 4, 2, 8, 1, 2)            \
  X(4, 4, 4, 8, 1, 2)

// exponent byte -> the power of two (255 -> NaN)
__device__ __forceinline__ float exp_scale(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7FC00000u : b == 0u ? 0x00400000u : b << 23);
}

// eight e2m1 codes times a power of two, exact in bf16 (2^128 and more, which only
// bytes 253 and 254 can give, become infinities)
__device__ __forceinline__ bf16x8 mx4x8_to_bf16(uint32_t c, float s) {
  u32x4 w;
  w.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
  w.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
  w.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
  w.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
  return __builtin_bit_cast(bf16x8, w);
}

__device__ __forceinline__ f32x4 mfma_bf16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// U: which byte of the scale words
template <int U>
__device__ __forceinline__ f32x4 mfma_mx4(const u32x4& a, const u32x4& b, const f32x4& c, uint32_t sa, uint32_t sb) {
  const u32x8 A = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const u32x8 B = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, A), __builtin_bit_cast(i32x8, B), c,
                                                          4, 4, U, (int)sa, U, (int)sb);
}

// WK: bf16 (false) or mx4 (true) weights; XK: the same of the activations
template <bool WK, bool XK, int NW, int R, int T, int D, int WPS>
__global__ __launch_bounds__(NW * 64, WPS) void experts_kernel(ExpertsDesc d, ExpertsArgs a, ExpertsPlan p) {
  static_assert(WK || !XK, "mx4 activations take mx4 weights");
  constexpr int kRows = 16 * T;
  constexpr uint32_t kStage = kRows * kStageBytes;       // a stage's rows in LDS
  constexpr uint32_t kScales = XK ? kRows * 16u : 0u;    // and their exponent bytes
  constexpr uint32_t kBuf = D * (kStage + kScales);
  constexpr int NL = WK && !XK ? 1 : 4;                  // 16-byte weight loads per row tile and stage
  constexpr int kLoads = R * (NL + (WK ? 1 : 0));        // weight loads per wave and stage
  constexpr int kWait = D * kLoads;                      // and of the whole ring
  static_assert(kWait < 64, "the wait fits the counter");
  // With one stage in the ring its copies are spread over the products of the
  // first quarter (in one go they hold up the LDS reads beside them, 12288 x
  // 5120 at 2048 rows 187 us instead of 181; over three quarters they land
  // later, gate/up of 8192 rows 286 instead of 281), its exponent bytes are
  // loaded a stage ahead, and so are weights that come in one load.
  constexpr bool kSpread = D == 1, kAhead = kSpread && NL == 1;
  constexpr int kYoung = kAhead ? 0 : kSpread ? 4 * R : kWait;  // weight loads after the last copy
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
  const int nst = (int)(XK ? (d.NU + 3) / 4 : d.NU);  // stages of K
  int lo, hi;
  split_range(nst, s, S, lo, hi);
  const int n = hi - lo;

  // ---- weights: this wave's row tiles (those past the last read zeros) ----
  const int64_t rt0 = (int64_t)rg * (NW * R) + wave * R;
  const int64_t nrt = d.NT - rt0 <= 0 ? 0 : d.NT - rt0 < R ? d.NT - rt0 : R;
  const __amdgpu_buffer_rsrc_t wr =
      make_rsrc(d.wpack + ((int64_t)e * d.NT + (nrt ? rt0 : 0)) * d.tile_bytes, (uint32_t)(nrt * d.tile_bytes));
  const uint32_t tb = (uint32_t)d.tile_bytes, so = (uint32_t)d.scale_off;
  u32x4 w[kAhead ? 2 : D][R][NL];
  uint32_t sc[kSpread ? 2 : D][WK ? R : 1];
  auto load_w = [&](auto slot, int r, int i, int c) __attribute__((always_inline)) {
    const int st = lo + c;
    uint32_t off = (uint32_t)r * tb;
    bool in = c < n;
    if constexpr (!WK) off += (uint32_t)st * 4096u + 1024u * i;
    else if constexpr (!XK) off += (uint32_t)st * 1024u;
    else {
      off += (uint32_t)(4 * st + i) * 1024u;
      in = in && 4 * st + i < (int)d.NU;
    }
    w[decltype(slot)::value][r][i] = buf_load16(wr, 16 * lane, in ? off : kOutOfRange);
  };
  auto load_s = [&](auto slot, int r, int c) __attribute__((always_inline)) {
    if constexpr (WK) {
      const int st = lo + c;
      const uint32_t off = (uint32_t)r * tb + so + (uint32_t)(XK ? st : st >> 2) * 256u;
      sc[decltype(slot)::value][r] = buf_load4(wr, 4 * lane, c < n ? off : kOutOfRange);
    }
  };

  auto load_scales = [&](auto slot, int c) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < R; ++r) load_s(slot, r, c);
  };

  // ---- activations.  A copy takes four rows x 256 bytes: lane l row l / 16,
  // piece (l % 16) ^ ((row - 4) % 16) of 16 bytes.  A read of 16 bytes a lane
  // serves 16 lanes at a time, rows 0-3 and 12-15 of one piece with rows 4-11 of
  // the next lane group's: with that shift they hit different banks for both
  // orders of the pieces (without it the bf16 x mx4 product reads at half
  // rate).  Rows past the group and bytes past the row take an offset beyond the
  // resource and land as zeros. ----
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
  // exponent bytes of mx4 activations: a copy takes 16 rows x 16 bytes
  constexpr int kSPer = XK ? (D * T + NW - 1) / NW : 1;
  uint32_t xso[kSPer];
  i32x4 xsr{};
  if constexpr (XK) {
    xsr = rsrc_words(a.xs + xrow0 * a.ldxs, (uint32_t)(xrows * a.ldxs));
#pragma unroll
    for (int i = 0; i < kSPer; ++i) {
      const uint32_t r = x_row(16 * ((wave + NW * i) % T) + (lane >> 2));
      xso[i] = r == 0xFFFFFFFFu ? kOutOfRange : r * (uint32_t)a.ldxs + 4u * (lane & 3);
    }
  }
  // copy number i (a compile-time index) of this wave's share of stages c ..
  // c + D - 1 of the split: first the rows, then the exponent bytes
  constexpr int kCopies = kPer + (XK ? kSPer : 0);
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
      const int id = wave + NW * (i - kPer), st = id / T, at = lo + c + st;
      if (D * T % NW == 0 || id < D * T)
        copy4<false>(xsr, buf + D * kStage + id * 256u, at >= hi ? kOutOfRange : xso[i - kPer],
                     (uint32_t)(at < hi ? at * 16 : 0));
    }
  };
  auto copy_x = [&](int c, uint32_t buf) __attribute__((always_inline)) {
    static_for<0, kCopies>([&](auto ic) __attribute__((always_inline)) { copy_one(c, buf, ic); });
  };

  // this lane's piece of row lane % 16 for step i
  const int fr = lane & 15;
  auto frag_off = [&](int i) __attribute__((always_inline)) -> uint32_t {
    const int pc = WK && !XK ? 4 * g + i : 4 * i + g;
    return (uint32_t)(fr * kStageBytes + 16 * (pc ^ ((fr - 4) & 15)));
  };
  uint32_t fo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) fo[i] = frag_off(i);

  f32x4 acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};

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
    if constexpr (!kSpread) {
      copy_x(c0 + D, other);
    }
    if constexpr (kSpread) load_scales(std::integral_constant<int, 1>{}, c0 + 1);
    if constexpr (kAhead) {
#pragma unroll
      for (int r = 0; r < R; ++r) load_w(std::integral_constant<int, 1>{}, r, 0, c0 + 1);
    }
    static_for<0, D>([&](auto sl) __attribute__((always_inline)) {
      constexpr int i = decltype(sl)::value;
      const int c = c0 + i;
      const uint8_t* xs = xb + cur + i * kStage;
      const uint8_t* xe = xb + cur + D * kStage + i * kScales;
      uint32_t sb[XK ? T : 1];
      if constexpr (XK) {
#pragma unroll
        for (int t = 0; t < T; ++t) sb[t] = *(const uint32_t*)(xe + t * 256 + fr * 16 + 4 * g);
      }
      float wsc[WK && !XK ? R : 1];
      if constexpr (WK && !XK) {
#pragma unroll
        for (int r = 0; r < R; ++r) wsc[r] = exp_scale((sc[i][r] >> (8 * ((lo + c) & 3))) & 255u);
      }
      // The stage's 4 T activation operands, in steps of one operand and its R
      // products; operands are read PF steps ahead of their products, and the
      // widened weights of a quarter are made during the quarter before.
      constexpr int PF = 4 * T > 8 ? 3 : 2;
      u32x4 b[PF + 1];
      auto read_b = [&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value;
        if constexpr (k < 4 * T) b[k % (PF + 1)] = *(const u32x4*)(xs + (k % T) * (16 * kStageBytes) + fo[k / T]);
      };
      bf16x8 A[2][R];
      auto widen = [&](auto qc, int r) __attribute__((always_inline)) {
        constexpr int q = decltype(qc)::value;
        if constexpr (!XK && q < 4) {
          if constexpr (WK) A[q & 1][r] = mx4x8_to_bf16(w[i][r][0][q], wsc[r]);
          else A[q & 1][r] = as_bf16x8(w[i][r][q]);
        }
      };
      static_for<0, PF>(read_b);
#pragma unroll
      for (int r = 0; r < R; ++r) widen(std::integral_constant<int, 0>{}, r);
      static_for<0, 4 * T>([&](auto kc) __attribute__((always_inline)) {
        constexpr int k = decltype(kc)::value, q = k / T, t = k % T;
        read_b(std::integral_constant<int, k + PF>{});
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if constexpr (XK) acc[r][t] = mfma_mx4<q>(w[i][r][q], b[k % (PF + 1)], acc[r][t], sc[i][r], sb[t]);
          else acc[r][t] = mfma_bf16(A[q & 1][r], as_bf16x8(b[k % (PF + 1)]), acc[r][t]);
        }
        if constexpr (!XK) {
#pragma unroll
          for (int r = t * R / T; r < (t + 1) * R / T; ++r) widen(std::integral_constant<int, q + 1>{}, r);
        }
        if constexpr (kSpread && k < T) {
          // past the last stage they write zeros: no branch in the loop
          static_for<k * kCopies / T, (k + 1) * kCopies / T>(
              [&](auto ic) __attribute__((always_inline)) { copy_one(c0 + D, other, ic); });
        }
        if constexpr (t == T - 1 && !kAhead) {
          // refill what this quarter was the last to read
          if constexpr (NL == 4) {
#pragma unroll
            for (int r = 0; r < R; ++r) load_w(sl, r, q, c + D);
          }
          if constexpr (q == 3) {
            if constexpr (NL == 1) {
#pragma unroll
              for (int r = 0; r < R; ++r) load_w(sl, r, 0, c + D);
            }
            if constexpr (!kSpread) load_scales(sl, c + D);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    });
    // the other buffer has landed and this one's reads are done
    ready(std::integral_constant<int, kYoung>{});
    if constexpr (kSpread && WK) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if constexpr (kAhead) w[0][r][0] = w[1][r][0];
        sc[0][r] = sc[1][r];
      }
    }
    cur = kBuf - cur;
  }
  SPENSE_WAIT_VM(0);

  static_assert(NW * kPartLds<R> <= 2 * kBuf, "the waves' parts of LDS");
  finish<R, T>(d, a, p, acc, xb + wave * kPartLds<R>, s, rg, j, rt0, row0, cnt, &last_flag);
}

template <bool WK, bool XK, int NW, int R, int T, int D, int WPS>
hipError_t launch_k(const ExpertsDesc& d, const ExpertsArgs& a, const ExpertsPlan& p, hipStream_t s) {
  const unsigned grid = grid_of(d, p, NW * R, NW * 64);
  if (!grid) return hipErrorInvalidValue;
  experts_kernel<WK, XK, NW, R, T, D, WPS><<<grid, NW * 64, 0, s>>>(d, a, p);
  return hipGetLastError();
}

template <bool WK, bool XK>
hipError_t launch_t(const ExpertsDesc& d, const ExpertsArgs& a, const ExpertsPlan& p, hipStream_t s) {
  switch (p.config) {
#define SPENSE_EXPERT_CASE(i, nw, r, t, dd, wps) \
  case i: return launch_k<WK, XK, nw, r, t, dd, wps>(d, a, p, s);
    SPENSE_EXPERT_CONFIGS(SPENSE_EXPERT_CASE)
#undef SPENSE_EXPERT_CASE
    default: return hipErrorInvalidValue;
  }
}

// Rows of bf16 into rows of ldo bytes, columns from K on zero, for rows whose
// length, stride or start is no whole number of 16 bytes, as the product's copies
// need them.  Eight columns a thread; bound by memory.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* X, int64_t M, int64_t K, int64_t ldx,
                                                       const int32_t* rows, int64_t R, uint8_t* out, int64_t ldo) {
  const uint32_t per = (uint32_t)(ldo / 16), id = blockIdx.x * 256u + threadIdx.x;  // at most 2^30 threads
  const uint32_t row = id / per;
  if (row >= R) return;
  const int64_t r = row, k = (int64_t)(id - row * per) * 8;
  const int64_t src = rows ? rows[r] : r;
  const bool in = src >= 0 && src < M;
  u32x4 o = u32x4{0, 0, 0, 0};
  if (in && k + 8 <= K) {
    o = *(const u32x4_any*)(X + src * ldx + k);
  } else if (in) {
    uint16_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = k + i < K ? X[src * ldx + k + i] : (uint16_t)0;
    o.x = v[0] | ((uint32_t)v[1] << 16);
    o.y = v[2] | ((uint32_t)v[3] << 16);
    o.z = v[4] | ((uint32_t)v[5] << 16);
    o.w = v[6] | ((uint32_t)v[7] << 16);
  }
  *(u32x4*)(out + r * ldo + 2 * k) = o;
}

}  // namespace

int experts_config_count() {
  int n = 0;
#define SPENSE_EXPERT_COUNT(i, nw, r, t, dd, wps) ++n;
  SPENSE_EXPERT_CONFIGS(SPENSE_EXPERT_COUNT)
#undef SPENSE_EXPERT_COUNT
  return n;
}

ExpertsShape experts_shape(int config) {
  switch (config) {
#define SPENSE_EXPERT_SHAPE(i, nw, r, t, dd, wps) \
  case i: return ExpertsShape{nw, r, t, dd};
    SPENSE_EXPERT_CONFIGS(SPENSE_EXPERT_SHAPE)
#undef SPENSE_EXPERT_SHAPE
    default: return ExpertsShape{0, 0, 0, 0};
  }
}

hipError_t launch_experts(const ExpertsDesc& d, const ExpertsArgs& a, int32_t xdtype, const ExpertsPlan& p,
                          hipStream_t s) {
  if (d.wdtype == DT_BF16) return xdtype == DT_BF16 ? launch_t<false, false>(d, a, p, s) : hipErrorInvalidValue;
  return xdtype == DT_MX4 ? launch_t<true, true>(d, a, p, s) : launch_t<true, false>(d, a, p, s);
}

hipError_t launch_pad_rows(const void* X, int64_t M, int64_t K, int64_t ldx, const int32_t* rows, int64_t R, void* out,
                           int64_t ldo, hipStream_t s) {
  // a launch's grid counts threads in 32 bits: runs of rows of at most 2^30
  const int64_t per = ldo / 16, most = (int64_t(1) << 30) / per;
  for (int64_t r = 0; r < R; r += most) {
    const int64_t n = R - r < most ? R - r : most;
    pad_rows_kernel<<<(unsigned)((n * per + 255) / 256), 256, 0, s>>>(
        (const uint16_t*)X + (rows ? 0 : r * ldx), rows ? M : n, K, ldx, rows ? rows + r : nullptr, n,
        (uint8_t*)out + r * ldo, ldo);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace spense
