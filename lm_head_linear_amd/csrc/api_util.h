// What the C-ABI entry points share: profiler ranges and the launcher.
#pragma once

#include <rocprofiler-sdk-roctx/roctx.h>

#include "flce_internal.h"

namespace flce {

// A named range around each entry point's call and each pass it enqueues
// (forward, merge, one per backward chunk or token chunk), for a profiler's
// marker trace (rocprofv3 --marker-trace). They span the host-side enqueue of
// the pass; the kernel trace gives the device times.
struct Range {
  explicit Range(const char* name) { roctxRangePushA(name); }
  ~Range() { roctxRangePop(); }
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

// The launcher of a call on `stream`, with the timing hooks while profiling.
Launcher make_launcher(void* stream);

}  // namespace flce
