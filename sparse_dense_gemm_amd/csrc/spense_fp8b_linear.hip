// HIP kernel of the products with packed block-scaled e4m3 weights (fp8b), for
// one weight matrix or a set of experts whose activation rows are grouped by
// expert in runs of any length.
//
//   Y[r, n] = sum_b sx[r, b] sw[n, b] sum_(k in b) x[r, k] w_e[n, k],   o_e <= r < o_(e+1),
//
// over blocks b of 128 columns.  The inner sum starts from zero and is added to
// the sums by a fused multiply-add with the product of the two scales, in 32
// bits: a scale that is no power of two cannot go through the matrix
// instruction's own scale operand, and rounding it into an operand would lose
// bits.  Three kinds of inner sums:
//   kBf16   bf16 x (sx = 1): four 16x16x32 products on the weights widened exactly
//           in registers;
//   kCodes  codes x, Y in bf16: one 16x16x128 product of codes.  The instruction
//           sums eight consecutive products at a time and drops what lies more than
//           13 bits below the largest of them (a product of 2^2 beside one of 2^16;
//           measured, and the same of 16x16x32 and with any operand as the eight);
//           on normal inputs that is 2e-5 of the result, a hundredth of the rounding
//           to bf16, for 3.5 times the rate of the 16x16x32 products (where large
//           products cancel it is more than that rounding: such callers take fp32);
//   kWide   codes x, Y in fp32: both widened to bf16, whose products and sums keep
//           the bits (6e-8 of the result).
// The scales cost four vector instructions to each 16x16x128, which takes the time
// of eight, so they run beside it.
//
// Tiles, launch order, split K and the way into Y are those of the products in
// spense_experts.hip: a workgroup owns NW R row tiles (16 R NW output columns)
// and up to 16 T activation rows of one expert; weights stream from memory into
// each wave's registers through a ring of D stages, activations are copied into
// LDS, D stages at a time into one of two buffers while the other is read.  A
// stage is 256 bytes of every row: 128 bf16 columns or 256 codes.
//
// What bounds it.  Few rows: the weights' way from memory (25600 x 5120 at one row
// 23 us, 5120 x 25600 at 29 rows 30 us: 5.6 and 4.5 TB/s).  Many rows of codes:
// operands from L2 and the matrix units in turn (55296 x 5120, 2048 rows 525 us,
// 2.2 PFLOP/s: matrix units busy 56% of the cycles, 75% where the loads are taken
// out, 394 us; 31 bytes a cycle and CU from L2; a plain library product of that size
// with one scale takes 466).  Many rows of bf16: the vector unit, which issues a
// 16x16x32 product (12 cycles of its time), two FMAs and half a widening in the 16
// cycles that the product runs (12288 x 5120, 2048 rows 214 us, 1.20 PFLOP/s; the
// library's bf16 product 241).  Experts: 16 x 3200 x 5120, 8192 rows of codes 161 us:
// 936 workgroups, two rounds of the 512 that run at once, where 1.8 would do.
#include "spense_experts_device.h"
#include "spense_fp8b.h"

namespace spense {
namespace {

// Configurations: X(index, waves, row tiles per wave R, m-tiles T, stages D in
// the ring and in an LDS buffer, waves per SIMD the registers allow).  The fewer
// m-tiles, the less there is to multiply behind a stage's loads and the more stages
// are on their way; the more row tiles a wave has, the more products an operand
// row read from LDS feeds.  us of configurations 0 to 4: 25600 x 5120 bf16 at one row
// 23, 27, 31, 43, -; 5120 x 25600 codes at 29 rows (fp32 out) 46, 32, 33, 45, -;
// 55296 x 5120 codes at 2048 rows -, -, 987, 662, 547; 12288 x 5120 bf16 there -, -,
// 327, 250, 229.
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
  X(4, 4, 4, 8, 1, 2)
// (256 columns of widened codes need more registers than two workgroups have)
#define SPENSE_FP8B_WIDE_CONFIGS(X) \
  X(0, 8, 1, 1, 8, 2)               \
  X(1, 4, 1, 2, 4, 2)               \
  X(2, 8, 1, 4, 2, 2)               \
  X(3, 4, 2, 8, 1, 2)

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

// POL: cache policy of the weights' loads
template <int KIND, int NW, int R, int T, int D, int WPS, int POL>
__global__ __launch_bounds__(NW * 64, WPS) void fp8b_kernel(Fp8bDesc d, Fp8bArgs a, ExpertsPlan p) {
  constexpr bool XQ = KIND != kBf16;                     // activations are codes
  constexpr int kRows = 16 * T;
  constexpr int NU = XQ ? 2 : 1;                         // units of a stage
  constexpr uint32_t kStage = kRows * kStageBytes;       // a stage's rows in LDS
  constexpr uint32_t kScales = XQ ? kRows * 8u : 0u;     // and their scales: [row][unit]
  constexpr uint32_t kBuf = D * (kStage + kScales);
  constexpr int NL = 2 * NU;                             // 16-byte weight loads per row tile and stage
  constexpr bool kSpread = D == 1;
  constexpr int kLoads = R * NL + (kSpread ? 0 : 1);     // with the weights' scales: vector loads per wave and stage
  constexpr int kWait = D * kLoads;                      // and of the whole ring
  static_assert(kWait < 64, "the wait fits the counter");
  // With one stage in the ring its copies are spread over the first products, and
  // its weights' scales, the same in every lane, are loaded a stage ahead into
  // scalar registers.
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
  const float* scales = d.scales + ((int64_t)e * d.SG + (nrt ? rt0 / 8 : 0)) * d.NUe * 2;
  const __amdgpu_buffer_rsrc_t sr = make_rsrc(scales, (uint32_t)(d.NUe * 8));
  const uint32_t tb = (uint32_t)d.tile_bytes;
  u32x4 w[D][R][NL];
  float sw[kSpread ? 2 : D][2 * NU];  // [unit][even, odd packed rows]
  // Piece i of row tile r for stage c: the stage's place is one scalar, chosen once
  // (beyond the resource past the last stage, and past the last unit for the
  // second unit's pieces), the row tile's a sum, the piece's a constant of the load.
  auto load_w = [&](auto slot, int r, int i, int c) __attribute__((always_inline)) {
    const int st = lo + c;
    const bool in = c < n && (!XQ || i < 2 || 2 * st + 1 < (int)d.NU);
    const uint32_t at = in ? (uint32_t)st * (NL * 1024u) : kOutOfRange;
    w[decltype(slot)::value][r][i] = buf_load16<POL>(wr, 16 * lane + 1024 * i, at + (uint32_t)r * tb);
  };
  auto load_scales = [&](auto slot, int c) __attribute__((always_inline)) {
    float(&o)[2 * NU] = sw[decltype(slot)::value];
    if constexpr (kSpread) {  // past the last stage the last one's again
      typedef const __attribute__((address_space(4))) float* Scalar;
      const Scalar p = (Scalar)(uintptr_t)(scales + (int64_t)(lo + (c < n ? c : n - 1)) * (2 * NU));
#pragma unroll
      for (int i = 0; i < 2 * NU; ++i) o[i] = p[i];
    } else {
      const uint32_t off = c < n ? (uint32_t)(lo + c) * (8u * NU) : kOutOfRange;
      if constexpr (XQ) {
        const f32x4 v = __builtin_bit_cast(f32x4, buf_load16(sr, 0, off));
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = v[i];
      } else {
        const f32x2 v = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(sr, 0, (int)off, 0));
        o[0] = v.x;
        o[1] = v.y;
      }
    }
  };

  // ---- activations.  In LDS a stage of an m-tile is four chunks of 64 bytes of
  // its 16 rows, one copy each: lane l brings row l / 4 and, of the chunk's four
  // pieces of 16 bytes, piece (l % 4) ^ f(row), f = 3 from row 8 on.  A read of 16
  // bytes a lane serves 16 lanes at a time, rows 0-3 and 12-15 of one lane group
  // with rows 4-11 of the next; with that shift they hit different banks where the
  // two groups' pieces are neighbours (codes) and where they are two apart (bf16).
  // A chunk needs no more than a lane's row to be addressed, so a wave that copies
  // two m-tiles keeps two offsets (four rows x 256 bytes a copy: eight, and four
  // for the reads, that the largest block does not have).  Rows past the group and
  // bytes past the row take an offset beyond the resource and land as zeros. ----
  constexpr int kPer = D * 4 * T / NW;                // copies of a buffer per wave
  constexpr int kTiles = T >= NW ? T / NW : 1;        // different m-tiles among them
  static_assert(T >= NW ? T % NW == 0 : NW % T == 0 && D % (NW / T) == 0, "every wave copies the same share");
  const int64_t xrow0 = a.rows ? 0 : row0;
  const int64_t xrows = a.rows ? a.M : cnt;
  const i32x4 xr = rsrc_words(a.X + xrow0 * a.ldx, (uint32_t)((xrows - 1) * a.ldx + a.xbytes));
  auto x_row = [&](int local) -> uint32_t {  // row of X behind row `local` of the group, or out of range
    if (local >= cnt) return 0xFFFFFFFFu;
    if (!a.rows) return (uint32_t)local;
    const int64_t q = a.rows[row0 + local];
    return q < 0 || q >= a.M ? 0xFFFFFFFFu : (uint32_t)q;
  };
  const int tile0 = T >= NW ? wave * kTiles : wave % T;
  const int piece = 16 * ((lane & 3) ^ (lane & 32 ? 3 : 0));  // bytes into the chunk
  const int limit = (int)a.xbytes - piece;  // of a chunk's place in the row
  uint32_t xo[kTiles];
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const uint32_t r = x_row(16 * (tile0 + i) + (lane >> 2));
    xo[i] = r == 0xFFFFFFFFu ? kOutOfRange : r * (uint32_t)a.ldx + (uint32_t)piece;
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
      constexpr int chunk = i % 4;
      const int tile = T >= NW ? tile0 + i / 4 : tile0;
      const int st = T >= NW ? 0 : wave / T + (NW / T) * (i / 4);
      const int at = lo + c + st;  // stage of K
      const int byte = at < hi ? at * kStageBytes + 64 * chunk : 0x7FFFFFFF;
      const uint32_t v = byte >= limit ? kOutOfRange : xo[T >= NW ? i / 4 : 0];
      copy16<false>(xr, buf + st * kStage + (4 * tile + chunk) * 1024u, v, (uint32_t)byte & 0x3FFFFFFFu);
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

  // this lane's piece of row lane % 16: codes, chunk 2 unit + half, piece g of it;
  // bf16, chunk 2 half + g / 2, pieces 2 (g % 2) and the next
  const int fr = lane & 15, shift = fr & 8 ? 3 : 0;
  const uint32_t fo = (uint32_t)(fr * 64 + (XQ ? 16 * (g ^ shift) : (g >> 1) * 1024 + 16 * ((2 * (g & 1)) ^ shift)));
  const uint32_t fo1 = XQ ? fo : fo ^ 16u;

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
      if constexpr (KIND == kCodes) {
        // 2 T steps of one operand and its R products; operands and their scales
        // are read a step ahead, a product's sum is taken kLag products later (55296
        // x 5120, 2048 rows: R = 4 one later 576 us, two 552, three 545; R = 2 one 678,
        // two 662)
        constexpr int kLag = R > 2 ? 3 : R, kRing = kLag + 1;
        static_assert(kLag <= R, "a sum is taken in its own step or the next, while its scales are there");
        const uint8_t* xe = xb + cur + D * kStage + i * kScales + fr * 8;
        u32x4 b[2][2];
        float sx[2], s0[2], s1[2];
        f32x4 P[kRing];
        auto read_b = [&](auto kc) __attribute__((always_inline)) {
          constexpr int k = decltype(kc)::value, q = k / T, t = k % T;
          if constexpr (k < 2 * T) {
            b[k & 1][0] = *(const u32x4*)(xs + fo + (4 * t + 2 * q) * 1024);
            b[k & 1][1] = *(const u32x4*)(xs + fo + (4 * t + 2 * q + 1) * 1024);
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
            __builtin_amdgcn_sched_barrier(0);
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
        // A unit goes in parts of QS operands (the whole one, or halves where the
        // registers are needed for sums: two vector instructions to a product
        // instead of one), each part in T steps of QS operands and their QS R
        // products, whose sums are taken in the next step.  The part's weights are
        // widened first, so that their registers are free for the loads of stage c + D.
        constexpr int QS = R * T >= 32 ? 2 : 4, kParts = NU * 4 / QS;
        constexpr int kFirst = T >= 4 ? T / 4 : 1;  // steps that the copies are spread over
        constexpr int kPieces = XQ ? QS / 2 : QS;   // 16-byte pieces of an operand row in LDS
        const uint8_t* xe = xb + cur + D * kStage + i * kScales + fr * 8;
        u32x4 b[2][kPieces];
        float sx[2];
        auto read_b = [&](auto kc) __attribute__((always_inline)) {
          constexpr int k = decltype(kc)::value, part = k / T, t = k % T, q0 = part * QS;  // q0: of 4 NU operands
          if constexpr (k < kParts * T) {
#pragma unroll
            for (int q = 0; q < kPieces; ++q)
              b[k & 1][q] = XQ ? *(const u32x4*)(xs + fo + (4 * t + q0 / 2 + q) * 1024)
                               : *(const u32x4*)(xs + ((q0 + q) & 1 ? fo1 : fo) + (4 * t + ((q0 + q) & 2)) * 1024);
            if constexpr (XQ) sx[k & 1] = *(const float*)(xe + t * 128 + 4 * (q0 / 4));
          }
        };
        read_b(std::integral_constant<int, 0>{});
        static_for<0, kParts>([&](auto pc) __attribute__((always_inline)) {
          constexpr int part = decltype(pc)::value, h0 = part * QS / 2, u = h0 / 2;  // h0: of 2 NU halves
          bf16x8 A[QS][R];
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < QS; ++q) {
              const u32x4& v = w[i][r][h0 + (q >> 1)];
              A[q][r] = q & 1 ? fp8x8_to_bf16(v.z, v.w) : fp8x8_to_bf16(v.x, v.y);
            }
          f32x4 P[R];
          float s0 = sw[i][2 * u], s1 = sw[i][2 * u + 1];
          static_for<0, T>([&](auto tc) __attribute__((always_inline)) {
            constexpr int t = decltype(tc)::value, k = part * T + t;
            read_b(std::integral_constant<int, k + 1>{});
            bf16x8 B[QS];
#pragma unroll
            for (int q = 0; q < QS; ++q) {
              if constexpr (XQ) {
                const u32x4& v = b[k & 1][q >> 1];
                B[q] = q & 1 ? fp8x8_to_bf16(v.z, v.w) : fp8x8_to_bf16(v.x, v.y);
              } else {
                B[q] = as_bf16x8(b[k & 1][q]);
              }
            }
            static_for<0, QS>([&](auto qc) __attribute__((always_inline)) {
              constexpr int q = decltype(qc)::value;
#pragma unroll
              for (int r = 0; r < R; ++r) {
                if constexpr (q == 0 && t > 0) add(acc[r][t - 1], P[r], s0, s1);
                P[r] = mfma_bf16(A[q][r], B[q], q == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : P[r]);
              }
            });
            if constexpr (XQ) {
              s0 = sx[k & 1] * sw[i][2 * u];
              s1 = sx[k & 1] * sw[i][2 * u + 1];
            }
            if constexpr (part == 0) copies(tc, std::integral_constant<int, kFirst>{});
            if constexpr (t == kFirst - 1) {
              static_for<0, QS / 2>([&](auto hc) __attribute__((always_inline)) {
#pragma unroll
                for (int r = 0; r < R; ++r) load_w(sl, r, h0 + decltype(hc)::value, c + D);
              });
            }
            __builtin_amdgcn_sched_barrier(0);
          });
#pragma unroll
          for (int r = 0; r < R; ++r) add(acc[r][T - 1], P[r], s0, s1);
        });
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

template <int KIND, int NW, int R, int T, int D, int WPS>
hipError_t launch_k(const Fp8bDesc& d, const Fp8bArgs& a, const ExpertsPlan& p, hipStream_t s) {
  const unsigned grid = grid_of(d, p, NW * R, NW * 64);
  if (!grid) return hipErrorInvalidValue;
  if constexpr (T < 8) {
    if (a.stream) {
      fp8b_kernel<KIND, NW, R, T, D, WPS, kNonTemporal><<<grid, NW * 64, 0, s>>>(d, a, p);
      return hipGetLastError();
    }
  }
  fp8b_kernel<KIND, NW, R, T, D, WPS, 0><<<grid, NW * 64, 0, s>>>(d, a, p);
  return hipGetLastError();
}

constexpr ExpertsShape kShapes[3][8] = {
#define SPENSE_FP8B_SHAPE(i, nw, r, t, dd, wps) {nw, r, t, dd},
    {SPENSE_FP8B_BF16_CONFIGS(SPENSE_FP8B_SHAPE)},
    {SPENSE_FP8B_CODES_CONFIGS(SPENSE_FP8B_SHAPE)},
    {SPENSE_FP8B_WIDE_CONFIGS(SPENSE_FP8B_SHAPE)},
#undef SPENSE_FP8B_SHAPE
};

}  // namespace

int fp8b_config_count(Fp8bKind kind) {
  int n = 0;
  while (n < 8 && kShapes[kind][n].waves) ++n;
  return n;
}

ExpertsShape fp8b_shape(Fp8bKind kind, int config) { return kShapes[kind][config]; }

hipError_t launch_fp8b_linear(const Fp8bDesc& d, const Fp8bArgs& a, const ExpertsPlan& p, hipStream_t s) {
#define SPENSE_FP8B_CASE(kind, i, nw, r, t, dd, wps) \
  case 8 * kind + i: return launch_k<kind, nw, r, t, dd, wps>(d, a, p, s);
#define SPENSE_FP8B_BF16_CASE(...) SPENSE_FP8B_CASE(kBf16, __VA_ARGS__)
#define SPENSE_FP8B_CODES_CASE(...) SPENSE_FP8B_CASE(kCodes, __VA_ARGS__)
#define SPENSE_FP8B_WIDE_CASE(...) SPENSE_FP8B_CASE(kWide, __VA_ARGS__)
  switch (8 * a.kind + p.config) {
    SPENSE_FP8B_BF16_CONFIGS(SPENSE_FP8B_BF16_CASE)
    SPENSE_FP8B_CODES_CONFIGS(SPENSE_FP8B_CODES_CASE)
    SPENSE_FP8B_WIDE_CONFIGS(SPENSE_FP8B_WIDE_CASE)
    default: return hipErrorInvalidValue;
  }
#undef SPENSE_FP8B_WIDE_CASE
#undef SPENSE_FP8B_CODES_CASE
#undef SPENSE_FP8B_BF16_CASE
#undef SPENSE_FP8B_CASE
}

}  // namespace spense
