// Optional per-launch timing (gns_timing_*), shared by the host sources.
#pragma once
#include <hip/hip_runtime.h>

namespace gns {

struct TimedLaunch {
  const char *name;
  const char *kernel;
  double flops, bytes;
  hipEvent_t start, stop;
};

// Brackets one launch with events while timing is enabled: construct before
// the launch, call done() after it.
struct LaunchScope {
  hipStream_t s;
  TimedLaunch rec{};
  bool on = false;
  LaunchScope(hipStream_t st, const char *name, const char *kernel, double flops, double bytes);
  void done();
};

}  // namespace gns
