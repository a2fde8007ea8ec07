// Host side of the mx4 and experts' layers: packing, launch planning,
// workspaces.  Arguments have been checked by the entry points in
// spense_api.cpp.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <new>

#include "../../include/spense.h"
#include "spense_mx.h"
#include "spense_workspace.h"

namespace spense {

struct ExpertsLayer {
  ExpertsDesc d{};
  int64_t weight_bytes = 0;
  int64_t device_bytes = 0;
  // workspaces, shared by the calls on the handle (one in flight)
  uint8_t* xws = nullptr;  // activations laid out for the product kernel
  size_t xws_bytes = 0;
  float* ws = nullptr;     // partial sums
  size_t ws_bytes = 0;
  int32_t* counters = nullptr;
  size_t n_counters = 0;
  GraphKept<kWorkspaces> graphs;  // workspaces that captured calls hold
  // rows that ws and counters have been sized for, whatever split count a
  // smaller call's plan takes: [mx4 activations][grouped]
  int64_t sized[2][2] = {{0, 0}, {0, 0}};
};

namespace {

constexpr int64_t kMaxPartials = int64_t(64) << 20;  // bytes of partial sums a plan may ask for
constexpr int kCUs = 256;

int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

int status_of(hipError_t e) {
  const int rc = report_hip(e);
  return e == hipErrorOutOfMemory ? SPENSE_ENOMEM : rc;
}

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

// Launch plan of R grouped rows (a function of ceil(R / 16) only, so that the
// workspaces of every smaller call can be sized by stepping over it): of the
// kernel's configurations and the split counts that fill one or two workgroups
// per CU, the one with the least estimated time.
ExpertsPlan make_plan(const ExpertsDesc& d, bool grouped, int64_t R, bool xmx) {
  // forced by SPENSE_EXPERTS=config[,splits[,rblock[,run]]] (tests, tuning)
  int f_config = -1, f_splits = 0, f_rblock = 0, f_run = 0;
  if (const char* v = getenv("SPENSE_EXPERTS")) {
    sscanf(v, "%d,%d,%d,%d", &f_config, &f_splits, &f_rblock, &f_run);
    if (f_config >= experts_config_count()) f_config = -1;
  }
  const int64_t R16 = (R + 15) / 16 * 16;
  const int64_t hit = grouped ? std::min(d.E, R16) : 1;  // experts that may have rows
  const int64_t rows = (R16 + hit - 1) / hit;            // rows of one, on average
  const int64_t stages = xmx ? (d.NU + 3) / 4 : d.NU;
  ExpertsPlan p{};
  double best = 0.0;
  for (int i = 0; i < experts_config_count(); ++i) {
    if (f_config >= 0 && i != f_config) continue;
    const ExpertsShape c = experts_shape(i);
    const int64_t per = c.waves * c.r, take = 16 * c.t;
    const int64_t rg = (d.NT + per - 1) / per;
    // sum over experts of ceil(n / take) for any split of R rows over `hit` experts
    const int64_t mg = grouped ? (R16 - hit) / take + hit : (R16 + take - 1) / take;
    // of them with rows: groups of no particular size leave half of their last m-group empty
    const double busy =
        grouped && hit > 1 ? (double)hit * std::max(1.0, (double)rows / (double)take + 0.5) : (double)mg;
    const int64_t most = std::min<int64_t>(std::max<int64_t>(1, stages / (xmx ? 2 : 4)), 64);
    int64_t tried = 0;
    for (int k = 0; k <= 2; ++k) {
      int64_t S = k == 0 ? 1 : std::min<int64_t>(most, (int64_t)(k * kCUs / ((double)rg * busy)));
      if (f_splits > 0) S = std::min<int64_t>(f_splits, std::min<int64_t>(stages, 64));
      while (S > 1 && S * d.NT * R16 * 64 > kMaxPartials) --S;
      if (S <= tried) continue;
      tried = S;
      const double t = plan_cycles(d, i, S, busy, hit, R16, xmx);
      if (best == 0.0 || t < best) {
        best = t;
        p.config = i;
        p.splits = (int)S;
        p.rgroups = (int)rg;
        p.mgroups = (int)mg;
      }
    }
  }
  const ExpertsShape c = experts_shape(p.config);
  // Launch order: large groups in blocks of four row groups, m-group by m-group
  // (the two workgroups of a CU, 32 apart, then share their row group's
  // weights), small ones, whose weights are most of what is read, m-group by
  // m-group of a single row group.
  p.rblock = f_rblock > 0 ? f_rblock : c.t >= 8 ? std::min(p.rgroups, 4) : 1;
  p.run = f_run;
  return p;
}

struct Need {
  int64_t xws = 0, ws = 0, cnt = 0;
  void grow(const Need& o) {
    xws = std::max(xws, o.xws);
    ws = std::max(ws, o.ws);
    cnt = std::max(cnt, o.cnt);
  }
};

Need plan_need(const ExpertsDesc& d, const ExpertsPlan& p, int64_t R) {
  Need n;
  if (p.splits > 1) {
    n.ws = (int64_t)p.splits * d.NT * ((R + 15) / 16 * 16) * 64;
    n.cnt = (int64_t)p.rgroups * p.mgroups;
  }
  return n;
}

bool fits(const ExpertsLayer* h, const Need& n) {
  return (int64_t)h->xws_bytes >= n.xws && (int64_t)h->ws_bytes >= n.ws && (int64_t)h->n_counters >= n.cnt;
}

// Replaces the workspaces that are too small (earlier launches may still use
// them, so the stream is synchronised first; those that a graph may hold stay).
int grow(ExpertsLayer* h, const Need& n, hipStream_t s) {
  hipError_t e = hipStreamSynchronize(s);
  if (e != hipSuccess) return status_of(e);
  auto regrow = [&](int which, void** p, size_t& have, int64_t want) -> int {
    if (want <= (int64_t)have) return SPENSE_OK;
    if (!h->graphs.drop(which, *p)) return SPENSE_ENOMEM;
    *p = nullptr;
    have = 0;
    const hipError_t err = hipMalloc(p, (size_t)want);
    if (err != hipSuccess) return status_of(err);
    have = (size_t)want;
    return SPENSE_OK;
  };
  int rc = regrow(kWsX, (void**)&h->xws, h->xws_bytes, n.xws);
  if (rc == SPENSE_OK) rc = regrow(kWsPartials, (void**)&h->ws, h->ws_bytes, n.ws);
  if (rc == SPENSE_OK && n.cnt > (int64_t)h->n_counters) {
    size_t bytes = h->n_counters * 4;
    rc = regrow(kWsCounters, (void**)&h->counters, bytes, n.cnt * 4);
    h->n_counters = bytes / 4;
    if (rc == SPENSE_OK) {
      e = launch_zero_i32(h->counters, n.cnt, s);
      if (e != hipSuccess) rc = status_of(e);
    }
  }
  return rc;
}

}  // namespace

void experts_release(ExpertsLayer* h) {
  if (!h) return;
  void* ptrs[] = {h->d.wpack, h->xws, h->ws, h->counters};
  for (void* p : ptrs)
    if (p) (void)hipFree(p);
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
  constexpr int64_t kSpan = int64_t(1) << 31;
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
  if (!fits(h, need)) {
    const int rc = grow(h, need, s);
    if (rc != SPENSE_OK) return rc;
  }
  sized = std::max(sized, R);
  if (need.xws || need.ws) h->graphs.used(s);
  hipError_t e = hipSuccess;
  a.M = M;
  if (prepare) {
    const int32_t* pick = gather ? rows : nullptr;
    if (xmx) {
      a.xs = h->xws + codes_bytes;
      e = launch_mx4_activations(X, M, d.K, ldx, pick, n_rows, h->xws, a.ldx, h->xws + codes_bytes, a.ldxs, s);
    } else {
      e = launch_pad_rows(X, M, d.K, ldx, pick, n_rows, h->xws, a.ldx, s);
    }
    if (e != hipSuccess) return status_of(e);
    a.X = h->xws;
    a.M = n_rows;
    if (gather) a.rows = nullptr;
  } else {
    a.X = (const uint8_t*)X;
  }
  a.ws = h->ws;
  a.counters = h->counters;
  e = launch_experts(d, a, xmx ? DT_MX4 : DT_BF16, p, s);
  return e == hipSuccess ? SPENSE_OK : status_of(e);
}

}  // namespace spense
