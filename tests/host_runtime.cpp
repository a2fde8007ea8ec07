// The host side of the library without a GPU: a runtime that hands out
// addresses (never touched) and remembers which are live, and launches that
// remember the pointers and row counts they were given.  Linked with the
// library's own host sources, so that tests can look at its workspaces.
#include <cstring>
#include <map>

#include "../sparse_dense_gemm_amd/csrc/spense_internal.h"
#include "../sparse_dense_gemm_amd/csrc/spense_mx.h"

namespace {

std::map<uint64_t, uint64_t> live;  // address -> bytes
uint64_t next_address = uint64_t(1) << 40;
int capturing = 0;

enum { X, PARTIALS, COUNTERS, X_ROWS, LAID_OUT, PICKED, ALLOCATIONS, FIELDS };
int64_t seen[FIELDS];

hipError_t saw(const void* x, const void* ws, const void* counters, int64_t rows) {
  seen[X] = (int64_t)x;
  seen[PARTIALS] = (int64_t)ws;
  seen[COUNTERS] = (int64_t)counters;
  seen[X_ROWS] = rows;
  return hipSuccess;
}

hipError_t laid_out(const int32_t* rows, int64_t n) {
  seen[LAID_OUT] = n;
  seen[PICKED] = rows != nullptr;
  return hipSuccess;
}

}  // namespace

extern "C" {

int64_t host_seen(int field) { return seen[field]; }
void host_forget(void) { std::memset(seen, 0, sizeof(seen)); }
void host_capturing(int on) { capturing = on; }
int host_live(int64_t p) { return live.count((uint64_t)p) != 0; }
int64_t host_live_bytes(void) {
  int64_t n = 0;
  for (const auto& e : live) n += (int64_t)e.second;
  return n;
}

hipError_t hipMalloc(void** p, size_t bytes) {
  ++seen[ALLOCATIONS];
  if (capturing) return hipErrorStreamCaptureUnsupported;
  *p = (void*)next_address;
  live[next_address] = bytes;
  next_address += (bytes + 4095) / 4096 * 4096 + 4096;
  return hipSuccess;
}
hipError_t hipFree(void* p) { return live.erase((uint64_t)p) ? hipSuccess : hipErrorInvalidValue; }
hipError_t hipStreamSynchronize(hipStream_t) { return capturing ? hipErrorStreamCaptureUnsupported : hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* st) {
  *st = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
  return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
  *d = 0;
  return hipSuccess;
}
hipError_t hipMemcpy(void*, const void*, size_t, hipMemcpyKind) { return hipSuccess; }
hipError_t hipMemcpyAsync(void*, const void*, size_t, hipMemcpyKind, hipStream_t) { return hipSuccess; }

}  // extern "C"

namespace spense {

// ---- mx4 and experts' layers (a table of shapes like the kernel's) ----
int experts_config_count() { return 5; }
ExpertsShape experts_shape(int i) {
  static const ExpertsShape t[5] = {{8, 1, 1, 8}, {4, 1, 2, 4}, {8, 1, 4, 2}, {4, 2, 8, 1}, {4, 4, 8, 1}};
  return t[i];
}
hipError_t launch_experts(const ExpertsDesc&, const ExpertsArgs& a, int32_t, const ExpertsPlan& p, hipStream_t) {
  return saw(a.X, p.splits > 1 ? a.ws : nullptr, p.splits > 1 ? a.counters : nullptr, a.M);
}
hipError_t launch_pad_rows(const void*, int64_t, int64_t, int64_t, const int32_t* rows, int64_t R, void*, int64_t,
                           hipStream_t) {
  return laid_out(rows, R);
}
hipError_t launch_mx4_activations(const void*, int64_t, int64_t, int64_t, const int32_t* rows, int64_t R, uint8_t*,
                                  int64_t, uint8_t*, int64_t, hipStream_t) {
  return laid_out(rows, R);
}
hipError_t launch_mx4_quantize(const void*, int32_t, int64_t, int64_t, int64_t, uint8_t*, int64_t, uint8_t*, int64_t,
                               hipStream_t) {
  return hipSuccess;
}
hipError_t launch_mx4_dequantize(const uint8_t*, int64_t, const uint8_t*, int64_t, int64_t, int64_t, void*, int32_t,
                                 int64_t, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_pack_experts(const ExpertsDesc&, const void*, int64_t, const uint8_t*, int64_t, hipStream_t) {
  return hipSuccess;
}
int64_t route_work_bytes(int64_t, int64_t) { return 0; }
hipError_t launch_route(const RouteArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_combine(const void*, int32_t, int64_t, int64_t, const int32_t*, const float*, int64_t, int64_t,
                          int64_t, void*, int32_t, int64_t, hipStream_t) {
  return hipSuccess;
}

// ---- sparse layers (no LDS-staged configurations) ----
int lds_preset_count() { return 0; }
LdsPreset lds_preset(int) { return LdsPreset{1, 1, 1, 1, 1}; }
int64_t lds_tile_bytes(int, int32_t, bool) { return int64_t(1) << 40; }
int lds_tile_copies(int, int32_t, bool) { return 1 << 20; }
hipError_t launch_pack(const LayerDesc&, const void*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t launch_export(const LayerDesc&, void*, uint32_t*, uint8_t*, void*, hipStream_t) { return hipSuccess; }
hipError_t launch_linear(const LayerDesc&, const LinearArgs& a, const LinearPlan&, hipStream_t) {
  return saw(a.X, a.ws, a.counters, a.M);
}
hipError_t launch_linear2(const LayerDesc&, const LinearArgs& a, const LinearPlan&, const LayerDesc&, const LinearArgs&,
                          const LinearPlan&, hipStream_t) {
  return saw(a.X, a.ws, a.counters, a.M);
}
hipError_t launch_zero_i32(int32_t*, int64_t, hipStream_t) { return hipSuccess; }
hipError_t scratch_area(hipStream_t, uint8_t**) { return hipErrorNotSupported; }
hipError_t launch_colsq(const void*, int64_t, int64_t, int64_t, float*, int64_t, float*, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_glu_scores(int32_t, const void*, const void*, int64_t, int64_t, int64_t, int64_t, const float*,
                             const float*, const float*, const float*, float*, float*, float*, float*, hipStream_t) {
  return hipSuccess;
}
hipError_t launch_rank_select(const float*, int64_t, int64_t, int*, uint8_t*, hipStream_t) { return hipSuccess; }
hipError_t launch_quantize_tokens(const void*, int64_t M, int64_t, int64_t, const int32_t*, int64_t, uint8_t*, int64_t,
                                  float*, hipStream_t) {
  return laid_out(nullptr, M);
}
hipError_t launch_gather_x(const LayerDesc&, const void*, int64_t M, int64_t, void*, hipStream_t) {
  return laid_out(nullptr, M);
}

}  // namespace spense
