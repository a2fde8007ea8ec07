// Entry points of the block-scaled e4m3 (fp8b) layers and of the norms around a
// block: argument checks, packing, launch planning, workspaces.
#include <algorithm>
#include <cmath>
#include <new>

#include "spense_fp8b.h"
#include "spense_layer.h"
#include "spense_product.h"

using namespace spense;

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 24, kMaxColumns = int64_t(1) << 20, kMaxExperts = 1024;
constexpr int64_t kMaxLd = int64_t(1) << 23;

bool float_type(int32_t t) { return t == SPENSE_F32 || t == SPENSE_BF16; }

// status of a type that has to be SPENSE_F32 or SPENSE_BF16
int float_status(int32_t t) {
  if (float_type(t)) return SPENSE_OK;
  return t == SPENSE_FP8_E4M3 || t == SPENSE_MX4 ? SPENSE_EUNSUPPORTED : SPENSE_EINVAL;
}

bool matrix_ok(int64_t M, int64_t K, int64_t ldc, int64_t lds) {
  return M >= 0 && M <= kMaxRows && K >= 1 && K <= kMaxColumns && ldc >= K && lds >= (K + kFp8Block - 1) / kFp8Block;
}

constexpr int64_t kKept = int64_t(96) << 20;

// Whether a launch's weights are streamed past the caches (configurations of fewer
// than 8 m-tiles have that form): where one m-group reads them (of experts' rows,
// which come in any number, where an average expert fills half of one), and they
// are more than a last-level cache that other layers share could keep.  us, default
// and streamed, layers in turn: 131 MB at one row 27.2 and 23.4, at 29 rows 32.9 and
// 29.0, at 64 rows 35.9 and 33.5; 262 MB of 16 experts, 128 rows 56.5 and 48.4, but
// 512 rows (two m-groups to some) 76 and 92; 66 MB at one row 14.0 and 15.5.
// R16: rows, rounded up to sixteen as the plan has them, so that a launch is the one
// that its plan priced.  Of few experts' rows less may be read than that counts: us
// of three layers of 16 experts, 262 MB each, in turn, one row 17.2 and 17.4, two
// 18.2 and 18.5, five 20.0 and 19.5, ten 23.5 and 22.3.
bool stream_weights(const Fp8bDesc& d, bool grouped, int64_t R16, const ExpertsShape& c) {
  const int64_t hit = grouped ? std::min(d.E, R16) : 1;
  if (c.t >= 8 || hit * d.NT * d.tile_bytes <= kKept) return false;
  return grouped && d.E > 1 ? R16 <= 8 * c.t * hit : R16 <= 16 * c.t;
}

// Estimated time of a launch of `groups` m-groups, in cycles or so.  Per stage (256
// bytes of every activation row) a workgroup multiplies and moves its weights and
// activations through the CU's vector cache; a stage takes at least the memory
// latency over the stages in flight, and the launch the time its weights take from
// memory, longer where they go through caches that do not keep them (131 MB at 29
// rows: 28 us streamed, 36 with two m-groups).  Two workgroups run together on a CU.
// With split K every sum is written and read once more, and a workgroup reads its
// tile's S sums by itself.  The constants are fitted to the order of 3678 timings
// (every configuration and split count that a plan may take, three kinds of
// products, 8 layers of 4 to 131 MB, 1 to 1024 rows): the plan's time is 1.010 of
// the best one's on average, at worst 1.15.
// Experts with few rows: fewer of them are hit than may be, in groups of any size,
// and workgroups of 128 columns then leave CUs idle, or read weights twice where an
// expert has more rows than they take; those of 64 columns (two m-tiles) spread
// better.  us of one, two and four m-tiles, gate/up of 16 experts of 3200 x 5120: 26
// rows of codes 36, 31, 33; 10 with fp32 out 23, 17, 30; 80 rows of codes 48, 36, 40,
// of bf16 45, 38, 44; of 1600 x 5120, 16 rows of bf16 23, 17, 28.  One m-tile of bf16,
// of which a CU takes two workgroups, is ahead where there are enough of them and
// experts have two rows or fewer: 10 rows 23, 27, 29.  Against every configuration, 45
// such layers of 4 to 700 tokens: 1.02 of the best one's time at the median, 1.14 at
// 90%, 1.25 at worst (149 tokens of bf16, 1600 x 5120: 28.4, one m-tile 22.7).
double plan_cycles(const Fp8bDesc& d, bool grouped, Fp8bKind kind, int config, int64_t S, double groups, int64_t hit,
                   int64_t R) {
  const ExpertsShape c = fp8b_shape(kind, config);
  const bool codes = kind != kBf16, few = grouped && d.E > 1 && groups <= (double)hit;
  if (few) groups *= 0.85;
  const double product = kind == kBf16 ? 10.4 : kind == kCodes ? 12.0 : 30.0;  // of a row tile and an m-tile
  const double more = c.t == 1 ? 1.7 : c.t == 2 ? 1.5 : c.t == 4 ? 1.42 : c.r == 2 ? 1.04 : 1.39;
  const double wkb = (codes ? 4.0 : 2.0) * c.waves * c.r, xkb = 4.0 * c.t;
  const double work = (product * c.waves * c.r * c.t + 15.0 * (wkb + xkb)) * more + 75.0;
  const double latency = c.stages > 1 ? 2400.0 / c.stages : 4150.0;
  const int64_t rg = (d.NT + c.waves * c.r - 1) / (c.waves * c.r);
  const int64_t stages = ((codes ? (d.NU + 1) / 2 : d.NU) + S - 1) / S;
  // a pass takes the ring's stages together; those past the end wait for nothing
  const int64_t empty = (stages + c.stages - 1) / c.stages * c.stages - stages;
  const int64_t load = (int64_t)std::ceil((double)rg * groups * (double)S / kCUs);  // workgroups of the fullest CU
  auto stage = [&](double w, double least) {
    return (double)(load / 2) * std::max(2.0 * w, least) + (load % 2 ? std::max(1.04 * w, least) : 0.0);
  };
  double t = stage(work, latency) * (double)stages + stage(0.5 * work, 0.0) * (double)empty;
  const int64_t bytes = hit * d.NT * d.tile_bytes;
  double memory = (double)bytes / (bytes <= kKept || stream_weights(d, grouped, R, c) ? 3260.0 : 2700.0);
  if (few) {
    const bool ahead = kind == kBf16 && R <= 2 * hit && (double)rg * groups >= kCUs;
    memory *= c.t == 1 && !ahead ? 1.06 : c.t <= 2 ? 0.85 : 0.94;
  }
  t = std::max(t, memory);
  t += 4000.0 * (double)((load + 1) / 2);
  if (S > 1) {
    const double tile = 1024.0 * c.waves * c.r * c.t;  // bytes of a workgroup's sums
    t += 4650.0 + (double)(S + 1) * tile / 80.0 + (double)(S * d.NT * 16 * R) * 8.0 / 1165.0;
  }
  return t;
}

ExpertsPlan make_plan(const Fp8bDesc& d, bool grouped, int64_t R, Fp8bKind kind) {
  const bool codes = kind != kBf16;
  return choose_plan(
      d, grouped, R, codes ? (d.NU + 1) / 2 : d.NU, codes ? 2 : 4, fp8b_config_count(kind),
      [&](int i) { return fp8b_shape(kind, i); },
      [&](int i, int64_t S, double groups, int64_t hit, int64_t R16) {
        return plan_cycles(d, grouped, kind, i, S, groups, hit, R16);
      },
      "SPENSE_FP8B");
}

// The activations of a call: bf16, or codes with their scales.
struct Activations {
  const void* X;
  int64_t ldx;
  const float* scales;  // codes only
  int64_t lds;
  bool quantize;        // bf16 that the call quantises
};

struct Fp8bLayer final : GroupedLayer {
  Fp8bDesc d{};
  int64_t weight_bytes = 0, device_bytes = 0;
  ProductWorkspaces w;
  // rows that the partial sums and counters have been sized for, whatever split
  // count a smaller call's plan takes and, with codes, whatever Y's type: [codes][grouped]
  int64_t sized[2][2] = {{0, 0}, {0, 0}};

  ~Fp8bLayer() override {
    if (d.wpack) (void)hipFree(d.wpack);
    if (d.scales) (void)hipFree(d.scales);
  }

  const ExpertsDesc& desc() const override { return d; }

  void info(spense_layer_info* info) const override {
    info->N = d.N;
    info->K = d.K;
    info->K_d = d.K;
    info->wdtype = d.wdtype;
    info->weight_bytes = weight_bytes;
    info->device_bytes = device_bytes;
    info->N_s = d.E;
    info->N_d = d.glu ? d.N / 2 : d.N;
  }

  int run(const void* X, int32_t adtype, int64_t M, int64_t ldx, const int32_t* rows, const int32_t* offsets,
          int64_t R, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s) override {
    return call(Activations{X, ldx, nullptr, 0, adtype == SPENSE_FP8_E4M3}, M, rows, offsets, R, Y, ydtype, ldy, s);
  }

  int call(const Activations& x, int64_t M, const int32_t* rows, const int32_t* offsets, int64_t R, void* Y,
           int32_t ydtype, int64_t ldy, hipStream_t s) {
    const bool grouped = offsets != nullptr, codes = x.quantize || x.scales;
    const Fp8bKind kind = !codes ? kBf16 : ydtype == SPENSE_F32 ? kWide : kCodes;
    const ExpertsPlan p = make_plan(d, grouped, R, kind);
    Fp8bArgs a{};
    a.rows = rows;
    a.offsets = offsets;
    a.R = R;
    a.Y = Y;
    a.ldy = ldy;
    a.ydtype = ydtype;
    a.kind = kind;
    a.stream = stream_weights(d, grouped, (R + 15) / 16 * 16, fp8b_shape(kind, p.config));
    // The product kernel reads rows of 16-byte pieces through offsets of 31
    // bits: activations are quantised into that form, or read in place if they
    // have it and laid out first if not: the R rows that are read, gathered if
    // they are picked by index, or X's own if it has no more than R and lies within
    // 31 bits.  So a call with fewer rows of X or in Y never needs a larger
    // workspace.
    const int64_t eb = x.scales ? 1 : 2, piece = 16 / eb;  // bytes of an element of X
    Need need = plan_need(d, p, R);
    bool prepare = true;
    if (!x.quantize) {
      const int64_t rows_span = rows ? M : 256;  // rows that one resource covers
      prepare = ((uintptr_t)x.X & 15) != 0 || x.ldx % piece != 0 || d.K % piece != 0 || x.ldx * eb * rows_span >= kSpan ||
                (x.scales && x.lds * 4 * rows_span >= kSpan);
    }
    if (!prepare) {
      a.ldx = x.ldx * eb;
      a.ldxs = x.lds * 4;
    } else {
      a.ldx = codes ? d.NU * kUnitK : (d.K + 7) / 8 * 16;
      a.ldxs = d.NU * 4;
    }
    a.xbytes = codes ? (prepare ? d.NU * kUnitK : d.K) : (d.K + 7) / 8 * 16;
    const bool gather = rows && (R < M || M * a.ldx >= kSpan);
    const int64_t n_rows = rows && !gather ? M : R;
    const int64_t codes_bytes = codes ? align256(n_rows * a.ldx) : 0;
    if (prepare) need.xws = codes ? codes_bytes + n_rows * a.ldxs : n_rows * a.ldx;
    int64_t& have = sized[codes][grouped];
    if (R > have) {  // every smaller call too: none of them may allocate later (graph capture)
      auto size = [&](int64_t r, Fp8bKind k) { need.grow(plan_need(d, make_plan(d, grouped, r, k), r)); };
      for (int64_t r = (have / 16 + 1) * 16; r < R + 16; r += 16) {
        const int64_t at = std::min(r, R);
        size(at, codes ? kCodes : kBf16);
        if (codes) size(at, kWide);
      }
    }
    if (!w.fits(need)) {
      const int rc = w.grow(need, s);
      if (rc != SPENSE_OK) return rc;
    }
    have = std::max(have, R);
    if (need.xws || need.ws) w.graphs.used(s);
    hipError_t e = hipSuccess;
    a.M = M;
    if (prepare) {
      const int32_t* pick = gather ? rows : nullptr;
      float* sx = (float*)(w.xws + codes_bytes);
      if (x.quantize) e = launch_fp8b_activations(x.X, M, d.K, x.ldx, pick, n_rows, w.xws, a.ldx, sx, d.NU, s);
      else if (codes)
        e = launch_fp8b_lay_out((const uint8_t*)x.X, x.ldx, x.scales, x.lds, M, d.K, pick, n_rows, w.xws, a.ldx, sx, d.NU,
                                s);
      else e = launch_pad_rows(x.X, M, d.K, x.ldx, pick, n_rows, w.xws, a.ldx, s);
      if (e != hipSuccess) return status_of(e);
      a.X = w.xws;
      a.xs = (const uint8_t*)sx;
      a.M = n_rows;
      if (gather) a.rows = nullptr;
    } else {
      a.X = (const uint8_t*)x.X;
      a.xs = (const uint8_t*)x.scales;
    }
    a.ws = w.ws;
    a.counters = w.counters;
    e = launch_fp8b_linear(d, a, p, s);
    return e == hipSuccess ? SPENSE_OK : status_of(e);
  }
};

int pack(const uint8_t* W, const float* scales, int64_t E, int64_t N, int64_t K, int64_t ldw, int64_t lds, int32_t glu,
         int split, void* stream, spense_handle* out) {
  Fp8bLayer* g = new (std::nothrow) Fp8bLayer();
  if (!g) return SPENSE_ENOMEM;
  const hipStream_t s = (hipStream_t)stream;
  Fp8bDesc& d = g->d;
  d.E = E;
  d.N = N;
  d.K = K;
  d.wdtype = SPENSE_FP8_E4M3;
  d.glu = glu ? 1 : 0;
  d.NT = (N + kRowTile - 1) / kRowTile;
  d.NU = mx_units(K);
  d.NUe = (d.NU + 1) / 2 * 2;
  d.SG = (d.NT + 7) / 8;
  d.tile_bytes = d.NU * 2048;
  const int64_t blocks = glu ? 2 * ((N / 2 + kFp8Block - 1) / kFp8Block) : (N + kFp8Block - 1) / kFp8Block;
  g->weight_bytes = E * (N * K + blocks * d.NU * 4);
  g->device_bytes = E * (d.NT * d.tile_bytes + d.SG * d.NUe * 8);
  spense_layer* h = new (std::nothrow) spense_layer();
  hipError_t e = h ? hipMalloc((void**)&d.wpack, (size_t)(E * d.NT * d.tile_bytes)) : hipErrorOutOfMemory;
  if (e != hipSuccess) d.wpack = nullptr;
  if (e == hipSuccess) {
    e = hipMalloc((void**)&d.scales, (size_t)(E * d.SG * d.NUe * 8));
    if (e != hipSuccess) d.scales = nullptr;
  }
  if (e == hipSuccess) e = launch_fp8b_pack(d, W, ldw, scales, lds, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) {
    (void)hipStreamSynchronize(s);
    delete g;
    delete h;
    return status_of(e);
  }
  h->split = split;
  h->grouped = g;
  *out = h;
  return SPENSE_OK;
}

// Codes and scales of activations: status, and the layer (split) of the handle.
int quantized_call(spense_handle h, const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int64_t M,
                   const int32_t* rows, const int32_t* offsets, int64_t R, void* Y, int32_t ydtype, int64_t ldy,
                   void* stream) {
  Fp8bLayer* g = static_cast<Fp8bLayer*>(h->grouped);
  const Fp8bDesc& d = g->d;
  if (ldc < d.K || lds < d.NU || ldy < (d.glu ? d.N / 2 : d.N)) return SPENSE_EINVAL;
  if (float_status(ydtype) != SPENSE_OK) return float_status(ydtype);
  if (ldc >= kMaxLd || lds >= kMaxLd) return SPENSE_EUNSUPPORTED;
  if (R == 0) return SPENSE_OK;
  return g->call(Activations{codes, ldc, scales, lds, false}, M, rows, offsets, R, Y, ydtype, ldy, (hipStream_t)stream);
}

bool finite(float v) { return std::fabs(v) <= 3.402823466e38f; }

}  // namespace

extern "C" {

int spense_quantize_fp8b(const void* X, int32_t xdtype, int64_t M, int64_t K, int64_t ldx, int32_t rows,
                         uint8_t* codes, int64_t ldc, float* scales, int64_t lds, void* stream) {
  if (!matrix_ok(M, K, ldc, lds) || ldx < K || (rows != 1 && rows != kFp8Block)) return SPENSE_EINVAL;
  if (M > 0 && (!X || !codes || !scales)) return SPENSE_EINVAL;
  if (float_status(xdtype) != SPENSE_OK) return float_status(xdtype);
  if (M == 0) return SPENSE_OK;
  // a row is read by several workgroups
  if (X == (const void*)codes || X == (const void*)scales || (const void*)codes == (const void*)scales)
    return SPENSE_EINVAL;
  const hipError_t e = launch_fp8b_quantize(X, xdtype, M, K, ldx, rows, codes, ldc, scales, lds, (hipStream_t)stream);
  return e == hipSuccess ? SPENSE_OK : report_hip(e);
}

int spense_dequantize_fp8b(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int32_t rows,
                           int64_t M, int64_t K, void* Y, int32_t ydtype, int64_t ldy, void* stream) {
  if (!matrix_ok(M, K, ldc, lds) || ldy < K || (rows != 1 && rows != kFp8Block)) return SPENSE_EINVAL;
  if (M > 0 && (!codes || !scales || !Y)) return SPENSE_EINVAL;
  if (float_status(ydtype) != SPENSE_OK) return float_status(ydtype);
  if (M == 0) return SPENSE_OK;
  if (Y == (const void*)codes || Y == (const void*)scales) return SPENSE_EINVAL;
  const hipError_t e = launch_fp8b_dequantize(codes, ldc, scales, lds, rows, M, K, Y, ydtype, ldy, (hipStream_t)stream);
  return e == hipSuccess ? SPENSE_OK : report_hip(e);
}

int spense_pack_fp8b(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int64_t N, int64_t K,
                     void* stream, spense_handle* out) {
  if (!out) return SPENSE_EINVAL;
  *out = nullptr;
  if (!codes || !scales || N < 1 || !matrix_ok(N, K, ldc, lds)) return SPENSE_EINVAL;
  return pack(codes, scales, 1, N, K, ldc, lds, 0, 5, stream, out);
}

int spense_linear_fp8b(spense_handle h, const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int64_t M,
                       void* Y, int32_t ydtype, int64_t ldy, void* stream) {
  if (!h || !codes || !scales || !Y || M < 1 || M > kMaxRows) return SPENSE_EINVAL;
  if (h->split != 5) return SPENSE_EUNSUPPORTED;
  return quantized_call(h, codes, ldc, scales, lds, M, nullptr, nullptr, M, Y, ydtype, ldy, stream);
}

int spense_pack_experts_fp8b(const uint8_t* W, const float* scales, int64_t E, int64_t N, int64_t K, int64_t ldw,
                             int64_t lds, int32_t glu, void* stream, spense_handle* out) {
  if (!out) return SPENSE_EINVAL;
  *out = nullptr;
  if (!W || !scales || E < 1 || E > kMaxExperts || N < 1 || (glu && N % 2) || !matrix_ok(N, K, ldw, lds))
    return SPENSE_EINVAL;
  return pack(W, scales, E, N, K, ldw, lds, glu, 6, stream, out);
}

int spense_experts_linear_fp8b(spense_handle h, const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds,
                               int64_t M, const int32_t* rows, const int32_t* offsets, int64_t R, void* Y,
                               int32_t ydtype, int64_t ldy, void* stream) {
  if (!h || !offsets || (R > 0 && (!codes || !scales || !Y))) return SPENSE_EINVAL;
  if (M < (R ? 1 : 0) || M > kMaxRows || R < 0 || R > kMaxRows || (!rows && M < R)) return SPENSE_EINVAL;
  if (h->split != 6) return SPENSE_EUNSUPPORTED;
  return quantized_call(h, codes, ldc, scales, lds, M, rows, offsets, R, Y, ydtype, ldy, stream);
}

int spense_block_norm(const spense_norm* n, void* stream) {
  if (!n || n->T < 0 || n->T > kMaxRows || n->H < 1 || n->H > kMaxColumns) return SPENSE_EINVAL;
  if (n->T > 0 && !n->Y && !n->residual_out) return SPENSE_EINVAL;
  if (!(n->eps >= 1.17549435e-38f) || !finite(n->eps) || !finite(n->scale)) return SPENSE_EINVAL;  // a normal number
  if (!n->pos != !n->weights) return SPENSE_EINVAL;
  if (n->pos && (n->k < 1 || n->k > kMaxExperts || n->O_rows < 0 || n->O_rows > kMaxRows)) return SPENSE_EINVAL;
  if (n->T > 0 && !n->O && !(n->pos && n->O_rows == 0)) return SPENSE_EINVAL;
  const bool codes = n->Y && n->ytype == SPENSE_FP8_E4M3;
  if (n->ldo < n->H || (n->gate && n->ldg != 0 && n->ldg < n->H) || (n->residual && n->ldr < n->H) ||
      (n->residual_out && n->ldro < n->H) || (n->Y && n->ldy < n->H))
    return SPENSE_EINVAL;
  if (codes ? (n->T > 0 && !n->yscales) || n->lds < (n->H + kFp8Block - 1) / kFp8Block : n->yscales != nullptr)
    return SPENSE_EINVAL;
  if (n->residual && n->residual == n->residual_out && n->ldr != n->ldro) return SPENSE_EINVAL;
  if (n->T > 0) {  // a row is read by several sums, and picked rows by several workgroups
    const void* const outs[] = {n->residual_out, n->Y, n->yscales};
    for (int i = 0; i < 3; ++i) {
      if (!outs[i]) continue;
      for (const void* in : {n->O, (const void*)n->pos, (const void*)n->weights, n->post, n->pre, n->gate})
        if (outs[i] == in) return SPENSE_EINVAL;
      if (i > 0 && outs[i] == n->residual) return SPENSE_EINVAL;  // the sum itself may take its place
      for (int j = 0; j < i; ++j)
        if (outs[i] == outs[j]) return SPENSE_EINVAL;
    }
  }
  const struct {
    bool used;
    int32_t type;
  } types[] = {{true, n->otype},
               {n->post || (n->pre && n->Y), n->wtype},
               {n->gate != nullptr, n->gtype},
               {n->residual || n->residual_out, n->rtype},
               {n->Y && !codes, n->ytype}};
  for (const auto& t : types)
    if (t.used && float_status(t.type) != SPENSE_OK) return float_status(t.type);
  if (n->T == 0) return SPENSE_OK;
  const hipError_t e = launch_block_norm(*n, (hipStream_t)stream);
  return e == hipSuccess ? SPENSE_OK : report_hip(e);
}

}  // extern "C"
