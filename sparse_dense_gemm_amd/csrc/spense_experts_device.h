// Device helpers shared by the products over grouped rows (spense_experts.hip,
// spense_fp8b_linear.hip): which tile a workgroup takes, the gate's SiLU, the
// way of a tile of sums into Y, and the grid that covers a plan.  Everything here
// is inline and file-local to each translation unit that includes it.
#pragma once

#include "spense_device.h"
#include "spense_mx.h"

namespace spense {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));  // at any element's address

// Groups of `rows` rows of the 64 experts from `base` on, lane i those of
// expert base + i: their number, and the number of those before and with them
// in this chunk; lo, hi: the expert's rows.
__device__ __forceinline__ int chunk_groups(const ExpertsDesc& d, const ExpertsArgs& a, int rows, int64_t base, int& lo,
                                            int& hi, int& incl) {
  const int lane = threadIdx.x & 63;
  const int64_t i = base + lane;
  int64_t l = 0, h = 0;
  if (i < d.E) {
    l = a.offsets[i];
    h = a.offsets[i + 1];
    l = l < 0 ? 0 : l > a.R ? a.R : l;
    h = h < l ? l : h > a.R ? a.R : h;
  }
  lo = (int)l;
  hi = (int)h;
  const int n = (hi - lo + rows - 1) / rows;
  incl = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  return n;
}

// Split, row group and m-group of this workgroup, of `groups` m-groups; false
// past the last tile.  Workgroups are dealt to the 8 XCDs round robin; the
// workgroups of an XCD take the tiles in runs, every XCD as many tiles, so that
// those running together there form a block of p.rblock row groups x some
// m-groups and share both operands in the XCD's L2 (gate/up of 8192 rows,
// 3200 x 5120 bf16: blocks of 2 to 4 row groups 275 us, of 7 280, of 13 288).
__device__ __forceinline__ bool tile_of(const ExpertsPlan& p, int groups, int& s, int& rg, int& j) {
  const uint32_t per = (uint32_t)p.rgroups * (uint32_t)groups, all = per * (uint32_t)p.splits;
  uint32_t run = (uint32_t)p.run;
  if (run == 0) {
    const uint32_t laps = (all + 511u) / 512u;
    run = laps ? (all + 8u * laps - 1u) / (8u * laps) : 1u;
  }
  const uint32_t b = blockIdx.x, xcd = b % 8u, seq = b / 8u, lap = seq / run;
  uint32_t id = (lap * 8u + xcd) * run + (seq - lap * run);
  if (id >= all) return false;
  s = 0;
  if (p.splits > 1) {
    s = (int)(id / per);
    id -= (uint32_t)s * per;
  }
  // blocks of rblock row groups (fewer in the last), one m-group after the other
  const uint32_t span = (uint32_t)p.rblock * (uint32_t)groups;
  const uint32_t blk = id / span, r0 = blk * (uint32_t)p.rblock, rem = id - blk * span;
  const uint32_t left = (uint32_t)p.rgroups - r0, nb = left < (uint32_t)p.rblock ? left : (uint32_t)p.rblock;
  const uint32_t m = rem / nb;
  j = (int)m;
  rg = (int)(r0 + rem - m * nb);
  return true;
}

// This workgroup's tile: split s, row group rg, m-group j, which is `cnt` rows
// of expert e from row0 on; false if it has none.  The m-groups are counted
// over the experts in order, so only those that have rows are dealt to the XCDs
// (dealing out every possible group left some XCDs with more of the real ones:
// 13 tokens' rows of mx4 gate/up 22.6 us, now 18.7; 8192 rows of mx4 down with
// its weighted sum 86.9, now 82.7).
__device__ __forceinline__ bool find_tile(const ExpertsDesc& d, const ExpertsArgs& a, const ExpertsPlan& p, int rows,
                                          int& s, int& rg, int& j, int& e, int64_t& row0, int& cnt) {
  if (!a.offsets) {
    if (!tile_of(p, (int)((a.R + rows - 1) / rows), s, rg, j)) return false;
    e = 0;
    row0 = (int64_t)j * rows;
    const int64_t left = a.R - row0;
    cnt = (int)(left < rows ? left : rows);
    return true;
  }
  int lo, hi, incl, groups = 0;
  int n = chunk_groups(d, a, rows, 0, lo, hi, incl);
  groups = __builtin_amdgcn_readlane(incl, 63);
  for (int64_t base = 64; base < d.E; base += 64) {
    chunk_groups(d, a, rows, base, lo, hi, incl);
    groups += __builtin_amdgcn_readlane(incl, 63);
  }
  // offsets that are not in order can name rows twice; the counters hold p.mgroups
  groups = groups < p.mgroups ? groups : p.mgroups;
  if (!tile_of(p, groups, s, rg, j)) return false;
  int before = 0;  // groups of the experts before this chunk of 64
  for (int64_t base = 0; base < d.E; base += 64) {
    if (d.E > 64) n = chunk_groups(d, a, rows, base, lo, hi, incl);
    const int excl = before + incl - n;
    const uint64_t hit = __ballot(j >= excl && j < excl + n);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int k = j - __builtin_amdgcn_readlane(excl, src);
      const int l0 = __builtin_amdgcn_readlane(lo, src), h0 = __builtin_amdgcn_readlane(hi, src);
      e = (int)base + src;
      row0 = (int64_t)(l0 + k * rows);
      const int left = h0 - (int)row0;
      cnt = left < rows ? left : rows;
      return cnt > 0;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// two fp32 as bf16, rounded to nearest even
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  bf16x2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

// silu(g) u.  The exponential and the reciprocal are the instructions; the
// product with log2(e) before the exponential is rounded, so the whole is within
// (|g| + 4) 2^-23 of itself.  The reciprocal instruction flushes results below
// the normal range, which 1 / (1 + exp(-g)) reaches at g = -87.3 before exp(-g)
// leaves the range of a float at -88.7, so both sides carry a quarter.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return 0.25f * g * __builtin_amdgcn_rcpf(fmaf(0.25f, __expf(-g), 0.25f)) * u;
}

// Sixteen activation rows of a wave's R row tiles into Y.  A lane holds four
// packed rows of each tile (v[r]), four output columns or two gated ones; its
// own stores would leave 32-byte runs, so the wave turns the block around in
// its part of LDS and writes each row's columns in runs of 16 bytes per lane.
// lds: 16 rows of at most 64 R + 16 bytes.  m0: Y row of the first of the
// `have` rows; col0: output column of the wave's first tile.
template <int R>
__device__ __forceinline__ void put_rows(const ExpertsDesc& d, const ExpertsArgs& a, const f32x4 (&v)[R], uint8_t* lds,
                                         int64_t m0, int have, int64_t col0) {
  const int lane = threadIdx.x & 63, fr = lane & 15, g = lane >> 4;
  const int eb = a.ydtype == DT_F32 ? 4 : 2;
  const int cols = d.glu ? 8 * R : 16 * R;           // output columns of the block
  const int64_t N = d.glu ? d.N / 2 : d.N;
  const int pitch = cols * eb + 16;
  uint8_t* row = lds + fr * pitch;
  asm volatile("" ::: "memory");  // the wave's own LDS accesses stay in this order
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (d.glu) {
      const float y0 = silu_mul(v[r][0], v[r][1]), y1 = silu_mul(v[r][2], v[r][3]);
      if (eb == 4) *(f32x2*)(row + (8 * r + 2 * g) * 4) = f32x2{y0, y1};
      else *(uint32_t*)(row + (8 * r + 2 * g) * 2) = bf16_pair(y0, y1);
    } else {
      if (eb == 4) *(f32x4*)(row + (16 * r + 4 * g) * 4) = v[r];
      else *(u32x2*)(row + (16 * r + 4 * g) * 2) = u32x2{bf16_pair(v[r][0], v[r][1]), bf16_pair(v[r][2], v[r][3])};
    }
  }
  asm volatile("" ::: "memory");
  const int lc = __builtin_ctz(cols * eb / 16);      // 16-byte pieces of a row: a power of two
  const int per = 16 / eb;
  for (int i = lane; i < (16 << lc); i += 64) {
    const int m = i >> lc, c = i & ((1 << lc) - 1);
    const int64_t col = col0 + c * per;
    if (m >= have || col >= N) continue;
    const uint8_t* from = lds + m * pitch + 16 * c;
    uint8_t* to = (uint8_t*)a.Y + ((m0 + m) * a.ldy + col) * eb;
    if (col + per <= N) {
      *(u32x4_any*)to = *(const u32x4*)from;
    } else {
      for (int k = 0; k < per && col + k < N; ++k) {
        if (eb == 4) ((uint32_t*)to)[k] = ((const uint32_t*)from)[k];
        else ((uint16_t*)to)[k] = ((const uint16_t*)from)[k];
      }
    }
  }
}

// LDS of a wave in put_rows
template <int R>
constexpr uint32_t kPartLds = 16 * (64 * R + 16);

// The end of a wave's R row tiles (rt0 ..) x T m-tiles (rows row0 .. row0 + cnt
// - 1 of Y): with split K the sums go to the workspace and the workgroup that
// arrives last adds them in split order.  Lane l holds the sums of packed rows
// 4 (l / 16) + 0..3 of a row tile at row l % 16 of an m-tile.  cnt may be zero
// or negative.
template <int R, int T>
__device__ __forceinline__ void finish(const ExpertsDesc& d, const ExpertsArgs& a, const ExpertsPlan& p,
                                       const f32x4 (&acc)[R][T], uint8_t* lds, int s, int rg, int j, int64_t rt0,
                                       int64_t row0, int cnt, int* last_flag) {
  const int lane = threadIdx.x & 63, fr = lane & 15, nb = 4 * (lane >> 4);
  const int S = p.splits;
  const __amdgpu_buffer_rsrc_t wsr = make_rsrc(a.ws, S > 1 ? (uint32_t)((int64_t)S * d.NT * a.R * 64) : 0u);
  auto poff = [&](int64_t split, int64_t rt, int64_t m) {
    return (uint32_t)((((split * d.NT + rt) * a.R + m) * 16 + nb) * 4);
  };
  if (S > 1) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t)
        if (rt0 + r < d.NT && 16 * t + fr < cnt) store_partial(wsr, poff(s, rt0 + r, row0 + 16 * t + fr), acc[r][t]);
    if (!arrive_last(a.counters + (int64_t)j * p.rgroups + rg, S, last_flag)) return;
  }
  if (rt0 >= d.NT) return;
#pragma unroll
  for (int t = 0; t < T; ++t) {
    if (16 * t >= cnt) break;
    const int64_t m = row0 + 16 * t + fr;
    f32x4 v[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      v[r] = acc[r][t];
      if (S > 1) {
        // in split order, eight at a time (one memory round trip per eight)
        v[r] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool in = rt0 + r < d.NT && 16 * t + fr < cnt;
        for (int s0 = 0; s0 < S; s0 += 8) {
          f32x4 part[8];
#pragma unroll
          for (int q = 0; q < 8; ++q)
            part[q] = load_partial(wsr, in && s0 + q < S ? poff(s0 + q, rt0 + r, m) : kOutOfRange);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (s0 + q < S) v[r] += part[q];
        }
      }
    }
    put_rows<R>(d, a, v, lds, row0 + 16 * t, cnt - 16 * t, rt0 * (d.glu ? 8 : 16));
  }
}

// grid of a plan, 0 if it does not fit: the workgroups of tile_of's runs for
// the largest number of m-groups (fewer m-groups never take more)
unsigned grid_of(const ExpertsDesc& d, const ExpertsPlan& p, int per, int threads) {
  if (p.rgroups != (d.NT + per - 1) / per || p.rblock < 1 || p.run < 0) return 0;
  const int64_t tiles = (int64_t)p.rgroups * p.mgroups * p.splits;
  const int64_t laps = (tiles + 511) / 512, run = p.run ? p.run : (tiles + 8 * laps - 1) / (8 * laps);
  const int64_t grid = (tiles + 8 * run - 1) / (8 * run) * (8 * run);
  return grid < 1 || grid * threads > 0x7FFFFFFF ? 0u : (unsigned)grid;  // threads count in 32 bits
}

}  // namespace
}  // namespace spense
