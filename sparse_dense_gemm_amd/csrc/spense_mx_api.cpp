// Host side of the mx4 and experts' layers: packing, launch planning,
// workspaces.  Arguments have been checked by the entry points in
// spense_api.cpp.
#include <algorithm>
#include <cmath>
#include <new>

#include "spense_product.h"

namespace spense {

struct ExpertsLayer {
  ExpertsDesc d{};
  int64_t weight_bytes = 0;
  int64_t device_bytes = 0;
  ProductWorkspaces w;
  // rows that ws and counters have been sized for, whatever split count a
  // smaller call's plan takes: [mx4 activations][grouped]
  int64_t sized[2][2] = {{0, 0}, {0, 0}};
};

namespace {

// Estimated cycles of a launch of `groups` m-groups.  Per stage (256 bytes of
// every activation row) a workgroup multiplies 4 waves r t operand pairs at 16
// cycles on each of four SIMDs and moves its weights and activations through
// the CU's vector cache at 64 bytes a cycle; the two hardly overlap (55296 x
// 5120 at 2048 rows: products alone 217 us, with the weights' or the rows'
// loads 261 and 247, with both 302).  A stage takes at least the memory latency over the stages
// in flight, and the launch the time its weights take from memory.  Two
// workgroups run together on a CU.  With split K every sum is written and read
// once more, and a workgroup reads its tile's S sums by itself.
double plan_cycles(const ExpertsDesc& d, int config, int64_t S, double groups, int64_t hit, int64_t R, bool xmx) {
  const ExpertsShape c = experts_shape(config);
  const bool mx = d.wdtype == SPENSE_MX4;
  const double wkb = (mx ? (xmx ? 4.25 : 1.25) : 4.0) * c.waves * c.r, xkb = 4.0 * c.t;
  // small m-tiles pay a barrier and their epilogue per fewer products
  const double work = (16.0 * c.waves * c.r * c.t + 16.0 * (wkb + xkb)) * (c.t < 4 ? 1.3 : c.t == 4 ? 1.45 : 1.0) + 60.0;
  // with one stage in the ring, weights of four loads wait behind its copies
  const double latency = c.stages > 1 ? 3000.0 / c.stages : mx && !xmx ? 2000.0 : 5000.0;
  const int64_t rg = (d.NT + c.waves * c.r - 1) / (c.waves * c.r);
  const int64_t stages = ((xmx ? (d.NU + 3) / 4 : d.NU) + S - 1) / S;
  // a pass takes the ring's stages together; those past the end wait for nothing
  const int64_t empty = (stages + c.stages - 1) / c.stages * c.stages - stages;
  const int64_t load = (int64_t)std::ceil((double)rg * groups * (double)S / kCUs);  // workgroups of the fullest CU
  auto stage = [&](double w, double least) {
    return (double)(load / 2) * std::max(2.0 * w, least) + (load % 2 ? std::max(1.3 * w, least) : 0.0);
  };
  double t = stage(work, latency) * (double)stages + stage(0.5 * work, 0.0) * (double)empty;
  t = std::max(t, (double)(hit * d.NT * d.tile_bytes) / 2600.0);
  t += 3000.0 * (double)((load + 1) / 2);
  if (S > 1) {
    const double tile = 1024.0 * c.waves * c.r * c.t;  // bytes of a workgroup's sums
    t += 4000.0 + (double)(S + 1) * tile / 40.0 + (double)(S * d.NT * 16 * R) * 8.0 / 1500.0;
  }
  return t;
}

ExpertsPlan make_plan(const ExpertsDesc& d, bool grouped, int64_t R, bool xmx) {
  return choose_plan(
      d, grouped, R, xmx ? (d.NU + 3) / 4 : d.NU, xmx ? 2 : 4, experts_config_count(), experts_shape,
      [&](int i, int64_t S, double groups, int64_t hit, int64_t R16) { return plan_cycles(d, i, S, groups, hit, R16, xmx); },
      "SPENSE_EXPERTS");
}

}  // namespace

void experts_release(ExpertsLayer* h) {
  if (!h) return;
  if (h->d.wpack) (void)hipFree(h->d.wpack);
  delete h;
}

int experts_pack(const void* W, int32_t wdtype, const uint8_t* scales, int64_t E, int64_t N, int64_t K, int64_t ldw,
                 int64_t lds, int32_t glu, hipStream_t s, ExpertsLayer** out) {
  ExpertsLayer* h = new (std::nothrow) ExpertsLayer();
  if (!h) return SPENSE_ENOMEM;
  ExpertsDesc& d = h->d;
  const bool mx = wdtype == SPENSE_MX4;
  d.E = E;
  d.N = N;
  d.K = K;
  d.wdtype = wdtype;
  d.glu = glu ? 1 : 0;
  d.NT = (N + kRowTile - 1) / kRowTile;
  d.NU = mx_units(K);
  d.scale_off = mx ? d.NU * 1024 : 0;
  d.tile_bytes = mx ? d.scale_off + (d.NU + 3) / 4 * 256 : d.NU * 4096;
  h->weight_bytes = mx ? E * N * ((K + 1) / 2 + (K + kMxBlock - 1) / kMxBlock) : E * N * K * 2;
  h->device_bytes = E * d.NT * d.tile_bytes;
  hipError_t e = hipMalloc((void**)&d.wpack, (size_t)h->device_bytes);
  if (e != hipSuccess) d.wpack = nullptr;
  if (e == hipSuccess) e = launch_pack_experts(d, W, ldw, scales, lds, s);
  if (e == hipSuccess) e = hipStreamSynchronize(s);
  if (e != hipSuccess) {
    (void)hipStreamSynchronize(s);
    experts_release(h);
    return status_of(e);
  }
  *out = h;
  return SPENSE_OK;
}

void experts_info(const ExpertsLayer* h, spense_layer_info* info) {
  info->N = h->d.N;
  info->K = h->d.K;
  info->K_d = h->d.K;
  info->wdtype = h->d.wdtype;
  info->weight_bytes = h->weight_bytes;
  info->device_bytes = h->device_bytes;
  info->N_s = h->d.E;
  info->N_d = h->d.glu ? h->d.N / 2 : h->d.N;
}

const ExpertsDesc& experts_desc(const ExpertsLayer* h) { return h->d; }

int experts_run(ExpertsLayer* h, const void* X, int32_t adtype, int64_t M, int64_t ldx, const int32_t* rows,
                const int32_t* offsets, int64_t R, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s) {
  const ExpertsDesc& d = h->d;
  const bool xmx = adtype == SPENSE_MX4;
  const ExpertsPlan p = make_plan(d, offsets != nullptr, R, xmx);
  ExpertsArgs a{};
  a.rows = rows;
  a.offsets = offsets;
  a.R = R;
  a.Y = Y;
  a.ldy = ldy;
  a.ydtype = ydtype;
  // The product kernel reads rows of 16-byte pieces through offsets of 31
  // bits: mx4 activations are quantised into that form, bf16 ones are read in
  // place if they have it and laid out first if not: the R rows that are read,
  // gathered if they are picked by index, or X's own if it has no more than R and
  // lies within 31 bits.  So a call with fewer rows of X or in Y never needs a
  // larger workspace.
  Need need = plan_need(d, p, R);
  bool prepare = true;
  if (xmx) {
    a.ldx = d.NU * 64;
    a.ldxs = (d.NU + 3) / 4 * 16;
    a.xbytes = a.ldx;
  } else {
    prepare = ((uintptr_t)X & 15) != 0 || ldx % 8 != 0 || d.K % 8 != 0 || 2 * ldx * 256 >= kSpan ||
              (rows && 2 * M * ldx >= kSpan);
    a.ldx = prepare ? (d.K + 7) / 8 * 16 : 2 * ldx;
    a.xbytes = (d.K + 7) / 8 * 16;
  }
  const bool gather = rows && (R < M || M * a.ldx >= kSpan);
  const int64_t n_rows = rows && !gather ? M : R;
  const int64_t codes_bytes = xmx ? align256(n_rows * a.ldx) : 0;
  if (prepare) need.xws = xmx ? codes_bytes + n_rows * a.ldxs : n_rows * a.ldx;
  int64_t& sized = h->sized[xmx][offsets != nullptr];
  if (R > sized) {  // every smaller call too: none of them may allocate later (graph capture)
    for (int64_t r = (sized / 16 + 1) * 16; r < R; r += 16) need.grow(plan_need(d, make_plan(d, offsets != nullptr, r, xmx), r));
  }
  if (!h->w.fits(need)) {
    const int rc = h->w.grow(need, s);
    if (rc != SPENSE_OK) return rc;
  }
  sized = std::max(sized, R);
  if (need.xws || need.ws) h->w.graphs.used(s);
  hipError_t e = hipSuccess;
  a.M = M;
  if (prepare) {
    const int32_t* pick = gather ? rows : nullptr;
    if (xmx) {
      a.xs = h->w.xws + codes_bytes;
      e = launch_mx4_activations(X, M, d.K, ldx, pick, n_rows, h->w.xws, a.ldx, h->w.xws + codes_bytes, a.ldxs, s);
    } else {
      e = launch_pad_rows(X, M, d.K, ldx, pick, n_rows, h->w.xws, a.ldx, s);
    }
    if (e != hipSuccess) return status_of(e);
    a.X = h->w.xws;
    a.M = n_rows;
    if (gather) a.rows = nullptr;
  } else {
    a.X = (const uint8_t*)X;
  }
  a.ws = h->w.ws;
  a.counters = h->w.counters;
  e = launch_experts(d, a, xmx ? DT_MX4 : DT_BF16, p, s);
  return e == hipSuccess ? SPENSE_OK : status_of(e);
}

}  // namespace spense
