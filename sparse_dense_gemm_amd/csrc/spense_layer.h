// The handle behind the C interface, shared by the files that implement its
// entry points (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "spense_internal.h"
#include "spense_mx.h"
#include "spense_workspace.h"

namespace spense {

// A packed layer over grouped rows whose code lives in a file of its own.  Status
// codes of spense.h; arguments have been checked by the entry points.
struct GroupedLayer {
  virtual ~GroupedLayer() {}
  virtual const ExpertsDesc& desc() const = 0;
  virtual void info(spense_layer_info* info) const = 0;
  // X: bf16 rows, quantised in the call if adtype is SPENSE_FP8_E4M3; offsets NULL: one expert takes all R rows
  virtual int run(const void* X, int32_t adtype, int64_t M, int64_t ldx, const int32_t* rows, const int32_t* offsets,
                  int64_t R, void* Y, int32_t ydtype, int64_t ldy, hipStream_t s) = 0;
};

}  // namespace spense

struct spense_layer {
  spense::LayerDesc d{};
  int device = 0;
  std::vector<int32_t> pi_host;
  uint8_t* wpack = nullptr;
  float* scales = nullptr;
  int32_t* pi = nullptr;
  int32_t* pip = nullptr;
  float* vals32 = nullptr;
  uint32_t* meta32 = nullptr;
  float* dense32 = nullptr;
  float* ws = nullptr;
  size_t ws_bytes = 0;
  void* xws = nullptr;  // activations in X'p order: gathered bf16 [M][K_p] (chunked staging of a chosen
                        // dense set), or W8A8 e4m3 codes [M][K_p] followed by the token scales [M]
  size_t xws_bytes = 0;
  int32_t* counters = nullptr;
  size_t n_counters = 0;
  spense::GraphKept<spense::kWorkspaces> graphs;  // workspaces that captured calls hold
  int32_t* ycol = nullptr;  // output column of each packed row, -1 on padding rows
  int32_t* wrow = nullptr;  // W row of each packed row (parts of an output-split layer)
  int64_t weight_bytes = 0;
  int64_t device_bytes = 0;
  // output-split layer (Technical Summary 2.A): no packed form of its own;
  // part[0] holds the 2:4 rows (no dense columns), part[1] the dense rows (no
  // sparse columns); either may be absent.  rho_host = [sparse rows | dense rows].
  // 0 input-split layer, 1 output-split layer, 2 GLU block, 3 mx4 layer, 4 experts' layers, 5 fp8b layer,
  // 6 fp8b experts' layers
  int split = 0;
  spense::ExpertsLayer* experts = nullptr;  // mx4 layer, experts' layers: their packed form
  spense::GroupedLayer* grouped = nullptr;  // fp8b layers: their packed form
  spense_layer* part[2] = {nullptr, nullptr};
  spense_layer* down = nullptr;  // GLU block: the down projection (input-split, read in rho order)
  int64_t N_s = 0, N_d = 0;
  std::vector<int32_t> rho_host;
};
