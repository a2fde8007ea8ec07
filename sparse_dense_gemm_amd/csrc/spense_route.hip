// HIP kernels of the expert router and of the weighted sum over a token's
// experts.
//
// Route: each token takes the k experts with the largest logits (NaN and -inf
// logits are never taken, equal ones go to the lower expert) with softmax
// weights, and the (token, choice) pairs are grouped by expert, in token order
// within an expert.  A token takes an expert at most once, so a bit per token
// and expert says everything about a block of tokens: an expert's rows in the
// block are the set bits, a token's place among them the set bits below its
// own.  The bits are set by LDS atomics whose order does not matter, so the
// result does not depend on it.  One launch for a single block of tokens, else
// two: the first leaves each block's counts in the workspace, the second adds
// up the counts of the blocks before its own.
#include <algorithm>

#include "spense_device.h"
#include "spense_mx.h"

namespace spense {
namespace {

// order-preserving bits of a logit; 0 for one that is never taken
__device__ __forceinline__ uint32_t logit_key(float l) {
  if (!(l > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(l + 0.0f);  // -0 becomes +0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float load_logit(const void* p, int32_t type, int64_t i) {
  return type == DT_F32 ? ((const float*)p)[i] : __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
}

// exp(l - max), also where both are +inf
__device__ __forceinline__ float weight_of(float l, float top) { return l == top ? 1.0f : expf(l - top); }

// Inclusive scan over the workgroup's threads (a multiple of 64 of them, at
// most 1024); tmp: 16 ints of LDS.
__device__ __forceinline__ int block_scan(int v, int* tmp) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(v, o);
    if (lane >= o) v += up;
  }
  if (lane == 63) tmp[wave] = v;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < wave; ++i) before += tmp[i];
  __syncthreads();
  return v + before;
}

// Largest value / smallest index over the G lanes that share a token.  Within
// rows of 16 lanes the operands move with the instruction (row rotations).
template <int CTRL>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  auto take = [&](uint32_t o) { v = o > v ? o : v; };
  take(row_ror<0x128>(v));
  take(row_ror<0x124>(v));
  take(row_ror<0x122>(v));
  take(row_ror<0x121>(v));
  if constexpr (G == 64) {
    take((uint32_t)__shfl_xor((int)v, 16));
    take((uint32_t)__shfl_xor((int)v, 32));
  }
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t group_min(uint32_t v) {
  return ~group_max<G>(~v);
}

constexpr int kHeld = 4096;  // choices of a block that are kept in LDS

// The choices of TB tokens.  G lanes share a token, V logits each; choice j is
// kept by lane j % G until the weights' sum is known.  With one block of tokens
// (fused) it also writes offsets, rows and final places; otherwise the block's
// counts and each choice's place within the block.  It reads every logit once
// and waits for little else than its own chain of k maxima: G lanes to a token
// keep it short (row rotations, no LDS), the least G and V that cover the
// experts leave no lane idle.  One token, 16 experts, 2 choices: 3.3 us; 8191
// tokens, 128 experts, 8 choices: 7.3 us, then 6.8 us of place_kernel.
template <int G, int V, int NT>
__global__ __launch_bounds__(NT) void choose_kernel(RouteArgs a, int TB, int fused) {
  extern __shared__ uint32_t bits[];  // [E][TB / 32], then (fused) [E] first rows
  __shared__ int tmp[16], last;
  __shared__ int16_t held[kHeld];
  const int words = TB / 32;
  const int E = (int)a.E;
  const bool hold = TB * a.k <= kHeld;
  for (int i = threadIdx.x; i < E * words; i += NT) bits[i] = 0u;
  __syncthreads();
  const int64_t t0 = (int64_t)blockIdx.x * TB;
  const int64_t left = a.T - t0;
  const int have = left < TB ? (int)left : TB;  // tokens of this block
  const int sub = threadIdx.x % G;
  constexpr int kTokens = NT / G;  // tokens at a time
  for (int tb = 0; tb < have; tb += kTokens) {
    const int tl = tb + threadIdx.x / G;
    const int64_t t = t0 + tl;
    const bool in = tl < have;
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = sub + G * v;
      key[v] = in && e < E ? logit_key(load_logit(a.logits, a.ltype, t * a.ldl + e)) : 0u;
    }
    // softmax over every expert that may be taken, if the weights are not
    // renormalised over the chosen ones
    float sum = 0.f, top = 0.f;
    if (!a.renormalize) {
      uint32_t m = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) m = key[v] > m ? key[v] : m;
      top = key_logit(group_max<G>(m));
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v]) sum += weight_of(key_logit(key[v]), top);
#pragma unroll
      for (int o = 1; o < G; o <<= 1) sum += __shfl_xor(sum, o, G);
    }
    for (int j0 = 0; j0 < a.k; j0 += G) {  // once for k <= G
      int my_e = -1;
      float my_w = 0.f;
      const int j1 = a.k - j0 < G ? a.k - j0 : G;
      for (int j = 0; j < j1; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) m = key[v] > m ? key[v] : m;
        m = group_max<G>(m);
        uint32_t e = 0xFFFFFFFFu;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
          if (key[v] == m) e = sub + G * v;  // equal keys: the lower expert
        e = group_min<G>(e);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e == (uint32_t)(sub + G * v)) key[v] = 0u;
        if (a.renormalize && j0 + j == 0) top = key_logit(m);
        if (m == 0u) break;
        if (sub == j) {
          my_e = (int)e;
          my_w = weight_of(key_logit(m), top);
        }
      }
      if (a.renormalize) {
        float s = my_w;
#pragma unroll
        for (int o = 1; o < G; o <<= 1) s += __shfl_xor(s, o, G);
        sum += s;
      }
      if (in && sub < j1) {
        const int64_t at = t * a.k + j0 + sub;
        a.ids[at] = my_e;
        a.weights[at] = a.renormalize && a.k > G ? my_w : my_e < 0 ? 0.f : my_w / sum;
        if (hold) held[tl * a.k + j0 + sub] = (int16_t)my_e;
        if (my_e >= 0) atomicOr(&bits[my_e * words + (tl >> 5)], 1u << (tl & 31));
      }
    }
    // more choices than lanes: the sum is known only now (a lane reads what it wrote)
    if (a.renormalize && a.k > G && in && sum > 0.f)
      for (int j = sub; j < a.k; j += G) a.weights[t * a.k + j] /= sum;
  }
  __syncthreads();
  // counts, and (fused) the experts' first rows
  int* first = (int*)(bits + E * words);
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += NT) {
    const int e = e0 + threadIdx.x;
    int n = 0;
    if (e < E)
      for (int i = 0; i < words; ++i) n += __popc(bits[e * words + i]);
    if (!fused) {
      if (e < E) a.work[(int64_t)blockIdx.x * E + e] = n;
    } else {
      const int incl = block_scan(n, tmp) + carry;
      if (e < E) {
        first[e] = incl - n;
        a.offsets[e] = incl - n;
        if (e == E - 1) a.offsets[E] = incl;
      }
      if (threadIdx.x == NT - 1) last = incl;
      __syncthreads();
      carry = last;
      __syncthreads();
    }
  }
  const int pairs = have * a.k;
  for (int i = threadIdx.x; i < pairs; i += NT) {
    const int tl = i / a.k;
    const int64_t at = t0 * a.k + i;
    const int e = hold ? held[i] : a.ids[at];
    int place = -1;
    if (e >= 0) {
      place = __popc(bits[e * words + (tl >> 5)] & ((1u << (tl & 31)) - 1u));
      for (int q = 0; q < (tl >> 5); ++q) place += __popc(bits[e * words + q]);
      if (fused) {
        place += first[e];
        a.rows[place] = (int)(t0 + tl);
      }
    }
    a.pos[at] = place;
  }
  if (fused)
    for (int64_t r = carry + threadIdx.x; r < a.T * a.k; r += NT) a.rows[r] = -1;
}

// Places of one block's choices: the counts of all blocks give the experts'
// first rows, those of the blocks before this one its own start among them.
// The threads split the blocks among them, P threads to an expert: what bounds
// it is the latency of a thread's reads in a row (8191 tokens, 128 experts: 62
// us of router with one thread to an expert and no reads ahead).
constexpr int kPlace = 1024;  // threads of place_kernel
__global__ __launch_bounds__(kPlace) void place_kernel(RouteArgs a, int TB, int blocks, int P) {
  extern __shared__ int base[];  // [E]
  __shared__ int tmp[16], last, all_s[kPlace], before_s[kPlace];
  const int E = (int)a.E;
  const int b = blockIdx.x;
  const int per = kPlace / P, part = threadIdx.x / per;  // experts at a time; share of the blocks
  int carry = 0;
  for (int e0 = 0; e0 < E; e0 += per) {
    const int e = e0 + threadIdx.x % per;
    int all = 0, before = 0;
    if (e < E) {
#pragma unroll 8
      for (int i = part; i < blocks; i += P) {
        const int n = a.work[(int64_t)i * E + e];
        all += n;
        before += i < b ? n : 0;
      }
    }
    all_s[threadIdx.x] = all;
    before_s[threadIdx.x] = before;
    __syncthreads();
    all = before = 0;
    if (part == 0)
      for (int q = 0; q < P; ++q) {
        all += all_s[threadIdx.x + q * per];
        before += before_s[threadIdx.x + q * per];
      }
    const int incl = block_scan(all, tmp) + carry;  // zeros beyond the first part
    if (part == 0 && e < E) {
      base[e] = incl - all + before;
      if (b == 0) {
        a.offsets[e] = incl - all;
        if (e == E - 1) a.offsets[E] = incl;
      }
    }
    if (threadIdx.x == kPlace - 1) last = incl;
    __syncthreads();
    carry = last;
    __syncthreads();
  }
  const int64_t t0 = (int64_t)b * TB, left = a.T - t0;
  const int pairs = (int)((left < TB ? left : TB) * a.k);
  for (int i = threadIdx.x; i < pairs; i += kPlace) {
    const int64_t at = t0 * a.k + i;
    const int e = a.ids[at];
    if (at >= carry) a.rows[at] = -1;  // rows past the last choice
    if (e < 0) continue;
    const int place = a.pos[at] + base[e];
    a.pos[at] = place;
    a.rows[place] = (int)(t0 + i / a.k);
  }
}

typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

// Y[t, n .. n + 3] = sum_j weights[t, j] O[pos[t, j], n .. n + 3], in the order
// of j.  Bound by memory (2048 tokens, 2 choices, 5120 columns f32 to bf16:
// 105 MB in 17.5 us, 6 TB/s); rows at any element's address move four columns
// at a time.
template <typename OT>
__global__ __launch_bounds__(256) void combine_kernel(const OT* O, int64_t R, int64_t ldo, const int32_t* pos,
                                                      const float* weights, int64_t T, int64_t k, int64_t N, void* Y,
                                                      int32_t ydtype, int64_t ldy) {
  const uint32_t per = (uint32_t)((N + 3) / 4), id = blockIdx.x * 256u + threadIdx.x;  // at most 2^30 threads
  const uint32_t row = id / per;
  const int64_t t = row, n = (int64_t)(id - row * per) * 4;
  if (t >= T) return;
  const bool full = n + 4 <= N;
  f32x4 y = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t j = 0; j < k; ++j) {
    const int64_t r = pos[t * k + j];
    if (r < 0 || r >= R) continue;
    const float w = weights[t * k + j];
    const OT* o = O + r * ldo + n;
    f32x4 v = f32x4{0.f, 0.f, 0.f, 0.f};
    if (full) {
      if constexpr (sizeof(OT) == 4) {
        v = *(const f32x4_any*)o;
      } else {
        const u32x2 u = *(const u32x2_any*)o;
        v = f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                  __uint_as_float(u.y & 0xFFFF0000u)};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) {
          if constexpr (sizeof(OT) == 4) v[i] = o[i];
          else v[i] = __uint_as_float((uint32_t)o[i] << 16);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] += w * v[i];
  }
  if (ydtype == DT_F32) {
    float* out = (float*)Y + t * ldy + n;
    if (full) *(f32x4_any*)out = y;
    else
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) out[i] = y[i];
  } else {
    uint16_t* out = (uint16_t*)Y + t * ldy + n;
    if (full) {
      u32x2 u;
      u.x = bf16_rne(y[0]) | (bf16_rne(y[1]) << 16);
      u.y = bf16_rne(y[2]) | (bf16_rne(y[3]) << 16);
      *(u32x2_any*)out = u;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) out[i] = (uint16_t)bf16_rne(y[i]);
    }
  }
}

__global__ void no_rows_kernel(int32_t* offsets, int64_t E) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i <= E) offsets[i] = 0;
}

// Tokens of a block.  Up to 256 tokens run as one block in one launch; more
// take the smallest blocks that leave at most 256 (each block reads every
// block's counts), as far as the bits take 48 KB of LDS.
int tokens_per_block(int64_t T, int64_t E) {
  if (T <= 256 && E * 32 <= 48 * 1024) return 256;
  int TB = 32;
  while (TB < 1024 && (T + TB - 1) / TB > 256 && E * (TB / 4) <= 48 * 1024) TB *= 2;
  return TB;
}

template <int G, int V>
hipError_t choose(const RouteArgs& a, int TB, int blocks, hipStream_t s) {
  const size_t lds = (size_t)a.E * (TB / 32) * 4 + (blocks == 1 ? (size_t)a.E * 4 : 0);
  // one block: 1024 threads where the tokens keep them busy
  if (blocks == 1 && a.T * G > 256) choose_kernel<G, V, 1024><<<1, 1024, lds, s>>>(a, TB, 1);
  else if (blocks == 1) choose_kernel<G, V, 256><<<1, 256, lds, s>>>(a, TB, 1);
  else choose_kernel<G, V, 512><<<blocks, 512, lds, s>>>(a, TB, 0);
  return hipGetLastError();
}

}  // namespace

// Counts of every block, for T tokens or any smaller number (whose blocks may
// be smaller and more).
int64_t route_work_bytes(int64_t T, int64_t E) {
  if (T <= tokens_per_block(T, E)) return 0;
  const int64_t blocks = (T + tokens_per_block(T, E) - 1) / tokens_per_block(T, E);
  return std::max(blocks, std::min<int64_t>((T + 31) / 32, 256)) * E * 4;
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.T == 0) {
    no_rows_kernel<<<(unsigned)((a.E + 256) / 256), 256, 0, s>>>(a.offsets, a.E);
    return hipGetLastError();
  }
  const int TB = tokens_per_block(a.T, a.E);
  const int blocks = (int)((a.T + TB - 1) / TB);
  hipError_t e;
  if (a.E <= 16) e = choose<16, 1>(a, TB, blocks, s);
  else if (a.E <= 32) e = choose<16, 2>(a, TB, blocks, s);
  else if (a.E <= 64) e = choose<16, 4>(a, TB, blocks, s);
  else if (a.E <= 128) e = choose<16, 8>(a, TB, blocks, s);
  else if (a.E <= 256) e = choose<16, 16>(a, TB, blocks, s);
  else if (a.E <= 512) e = choose<64, 8>(a, TB, blocks, s);
  else e = choose<64, 16>(a, TB, blocks, s);
  if (e != hipSuccess || blocks == 1) return e;
  int P = 1;  // threads to an expert: all of them at work
  while (P < 64 && a.E * 2 * P <= kPlace) P *= 2;
  place_kernel<<<blocks, kPlace, (size_t)a.E * 4, s>>>(a, TB, blocks, P);
  return hipGetLastError();
}

hipError_t launch_combine(const void* O, int32_t otype, int64_t R, int64_t ldo, const int32_t* pos,
                          const float* weights, int64_t T, int64_t k, int64_t N, void* Y, int32_t ydtype, int64_t ldy,
                          hipStream_t s) {
  const int64_t per = (N + 3) / 4, most = (int64_t(1) << 30) / per;  // a grid counts threads in 32 bits
  const int yb = ydtype == DT_F32 ? 4 : 2;
  for (int64_t t = 0; t < T; t += most) {
    const int64_t n = T - t < most ? T - t : most;
    const unsigned grid = (unsigned)((n * per + 255) / 256);
    void* y = (uint8_t*)Y + t * ldy * yb;
    if (otype == DT_F32)
      combine_kernel<float><<<grid, 256, 0, s>>>((const float*)O, R, ldo, pos + t * k, weights + t * k, n, k, N, y,
                                                 ydtype, ldy);
    else
      combine_kernel<uint16_t><<<grid, 256, 0, s>>>((const uint16_t*)O, R, ldo, pos + t * k, weights + t * k, n, k, N,
                                                    y, ydtype, ldy);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace spense
