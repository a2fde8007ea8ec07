// Failures for the host library of host_runtime.cpp, by the linker's --wrap: the
// zeroing launch or an allocation fails when it is told to.
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {
int zero_fails = 0;       // zeroing launches that fail from now on
int64_t zeroed = 0;       // address that was zeroed last
int64_t alloc_fails = 0;  // allocations of this many bytes or more fail, once
hipError_t last = hipSuccess;  // kept until it is asked for, as the runtime does
}  // namespace

extern "C" {

void host_fail_zero(int n) { zero_fails = n; }
int64_t host_zeroed(void) { return zeroed; }
void host_fail_alloc(int64_t bytes) { alloc_fails = bytes; }

int host_last_error(void) { return (int)last; }
hipError_t __wrap_hipGetLastError(void) {
  const hipError_t e = last;
  last = hipSuccess;
  return e;
}

hipError_t __real_hipMalloc(void** p, size_t bytes);
hipError_t __wrap_hipMalloc(void** p, size_t bytes) {
  if (alloc_fails && (int64_t)bytes >= alloc_fails) {
    alloc_fails = 0;
    return last = hipErrorOutOfMemory;
  }
  return __real_hipMalloc(p, bytes);
}

// spense::launch_zero_i32(int32_t*, int64_t, hipStream_t)
hipError_t __wrap__ZN6spense15launch_zero_i32EPilP12ihipStream_t(int32_t* p, int64_t, hipStream_t) {
  if (zero_fails > 0) {
    --zero_fails;
    return last = hipErrorLaunchFailure;
  }
  zeroed = (int64_t)p;
  return hipSuccess;
}

}  // extern "C"
