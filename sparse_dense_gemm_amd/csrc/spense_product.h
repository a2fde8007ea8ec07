// Host code shared by the products over grouped rows (spense_mx_api.cpp,
// spense_fp8b_api.cpp): launch planning and a handle's workspaces.
#pragma once

#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "../../include/spense.h"
#include "spense_internal.h"
#include "spense_mx.h"
#include "spense_workspace.h"

namespace spense {

constexpr int64_t kMaxPartials = int64_t(64) << 20;  // bytes of partial sums a plan may ask for
constexpr int kCUs = 256;
constexpr int64_t kSpan = int64_t(1) << 31;          // the product kernels' offsets have 31 bits

inline int64_t align256(int64_t n) { return (n + 255) / 256 * 256; }

inline int status_of(hipError_t e) {
  const int rc = report_hip(e);
  return e == hipErrorOutOfMemory ? SPENSE_ENOMEM : rc;
}

// Launch plan of R grouped rows (a function of ceil(R / 16) only, so that the
// workspaces of every smaller call can be sized by stepping over it): of the
// kernel's configurations and the split counts that fill one or two workgroups
// per CU, the one with the least estimated time.
//   stages     stages of K; a split has at least `least` of them
//   shape(i)   configuration i of `configs`
//   cycles(i, S, groups, hit, R16)  estimated cycles of a launch
//   forced     name of an environment variable with config[,splits[,rblock[,run]]] (tests, tuning)
template <typename Shape, typename Cycles>
ExpertsPlan choose_plan(const ExpertsDesc& d, bool grouped, int64_t R, int64_t stages, int64_t least, int configs,
                        Shape&& shape, Cycles&& cycles, const char* forced) {
  int f_config = -1, f_splits = 0, f_rblock = 0, f_run = 0;
  if (const char* v = getenv(forced)) {
    sscanf(v, "%d,%d,%d,%d", &f_config, &f_splits, &f_rblock, &f_run);
    if (f_config >= configs) f_config = -1;
  }
  const int64_t R16 = (R + 15) / 16 * 16;
  const int64_t hit = grouped ? std::min(d.E, R16) : 1;  // experts that may have rows
  const int64_t rows = (R16 + hit - 1) / hit;            // rows of one, on average
  ExpertsPlan p{};
  double best = 0.0;
  for (int i = 0; i < configs; ++i) {
    if (f_config >= 0 && i != f_config) continue;
    const ExpertsShape c = shape(i);
    const int64_t per = c.waves * c.r, take = 16 * c.t;
    const int64_t rg = (d.NT + per - 1) / per;
    // sum over experts of ceil(n / take) for any split of R rows over `hit` experts
    const int64_t mg = grouped ? (R16 - hit) / take + hit : (R16 + take - 1) / take;
    // of them with rows: groups of no particular size leave half of their last m-group empty
    const double busy =
        grouped && hit > 1 ? (double)hit * std::max(1.0, (double)rows / (double)take + 0.5) : (double)mg;
    const int64_t most = std::min<int64_t>(std::max<int64_t>(1, stages / least), 64);
    int64_t tried = 0;
    for (int k = 0; k <= 2; ++k) {
      int64_t S = k == 0 ? 1 : std::min<int64_t>(most, (int64_t)(k * kCUs / ((double)rg * busy)));
      if (f_splits > 0) S = std::min<int64_t>(f_splits, std::min<int64_t>(stages, 64));
      while (S > 1 && S * d.NT * R16 * 64 > kMaxPartials) --S;
      if (S <= tried) continue;
      tried = S;
      const double t = cycles(i, S, busy, hit, R16);
      if (best == 0.0 || t < best) {
        best = t;
        p.config = i;
        p.splits = (int)S;
        p.rgroups = (int)rg;
        p.mgroups = (int)mg;
      }
    }
  }
  const ExpertsShape c = shape(p.config);
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

inline Need plan_need(const ExpertsDesc& d, const ExpertsPlan& p, int64_t R) {
  Need n;
  if (p.splits > 1) {
    n.ws = (int64_t)p.splits * d.NT * ((R + 15) / 16 * 16) * 64;
    n.cnt = (int64_t)p.rgroups * p.mgroups;
  }
  return n;
}

// Workspaces of a handle, shared by its calls (one in flight).
struct ProductWorkspaces {
  uint8_t* xws = nullptr;  // activations laid out for the product kernel
  size_t xws_bytes = 0;
  float* ws = nullptr;     // partial sums
  size_t ws_bytes = 0;
  int32_t* counters = nullptr;
  size_t n_counters = 0;
  GraphKept<kWorkspaces> graphs;  // workspaces that captured calls hold

  ProductWorkspaces() = default;
  ProductWorkspaces(const ProductWorkspaces&) = delete;
  ProductWorkspaces& operator=(const ProductWorkspaces&) = delete;
  ~ProductWorkspaces() {
    void* ptrs[] = {xws, ws, counters};
    for (void* p : ptrs)
      if (p) (void)hipFree(p);
  }

  bool fits(const Need& n) const {
    return (int64_t)xws_bytes >= n.xws && (int64_t)ws_bytes >= n.ws && (int64_t)n_counters >= n.cnt;
  }

  // Replaces the workspaces that are too small (earlier launches may still use
  // them, so the stream is synchronised first; those that a graph may hold stay).
  // One that cannot be replaced stays as it is, and so does what it suffices for.
  int grow(const Need& n, hipStream_t s) {
    hipError_t e = hipStreamSynchronize(s);
    if (e != hipSuccess) return status_of(e);
    auto regrow = [&](int which, void** p, size_t& have, int64_t want, auto&& fill) -> int {
      if (want <= (int64_t)have) return SPENSE_OK;
      void* fresh = nullptr;
      hipError_t err = hipMalloc(&fresh, (size_t)want);
      if (err != hipSuccess) return status_of(err);
      err = fill(fresh);
      if (err != hipSuccess || !graphs.drop(which, *p)) {
        (void)hipFree(fresh);
        return err == hipSuccess ? SPENSE_ENOMEM : status_of(err);
      }
      *p = fresh;
      have = (size_t)want;
      return SPENSE_OK;
    };
    auto as_is = [](void*) { return hipSuccess; };
    int rc = regrow(kWsX, (void**)&xws, xws_bytes, n.xws, as_is);
    if (rc == SPENSE_OK) rc = regrow(kWsPartials, (void**)&ws, ws_bytes, n.ws, as_is);
    size_t bytes = n_counters * 4;
    if (rc == SPENSE_OK)
      rc = regrow(kWsCounters, (void**)&counters, bytes, n.cnt * 4,
                  [&](void* p) { return launch_zero_i32((int32_t*)p, n.cnt, s); });
    n_counters = bytes / 4;
    return rc;
  }
};

}  // namespace spense
