// What the fp8b products' launches are told, for the host library of
// host_runtime.cpp (by the linker's --wrap).
#include "../sparse_dense_gemm_amd/csrc/spense_fp8b.h"

namespace {
int64_t told[4];  // weights streamed, configuration, splits, launches
}

extern "C" {

int64_t host_told(int field) { return told[field]; }

// spense::launch_fp8b_linear(const Fp8bDesc&, const Fp8bArgs&, const ExpertsPlan&, hipStream_t)
hipError_t __wrap__ZN6spense18launch_fp8b_linearERKNS_8Fp8bDescERKNS_8Fp8bArgsERKNS_11ExpertsPlanEP12ihipStream_t(
    const spense::Fp8bDesc&, const spense::Fp8bArgs& a, const spense::ExpertsPlan& p, hipStream_t) {
  told[0] = a.stream;
  told[1] = p.config;
  told[2] = p.splits;
  ++told[3];
  return hipSuccess;
}

}  // extern "C"
