// Argument checks and stage events shared by the C ABI's entry points.
#pragma once

#include <math.h>
#include <stdint.h>

#include "kernels.h"

#include "../../include/topmoe.h"

namespace topmoe {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Stage i's launch: the stream plus, when timing is requested, events
// 2i / 2i+1 stamped by the stage's kernel dispatch.
struct Stages {
  void* const* ev;
  hipStream_t s;
  Launch at(int i) const {
    Launch L;
    L.s = s;
    if (ev) {
      L.start = static_cast<hipEvent_t>(ev[2 * i]);
      L.stop = static_cast<hipEvent_t>(ev[2 * i + 1]);
    }
    return L;
  }
  // A stage that enqueued no kernel still gets both events (zero length).
  hipError_t close(const Launch& L) const {
    if (!ev || L.launched) return hipSuccess;
    const hipError_t e = hipEventRecord(L.start, s);
    return e != hipSuccess ? e : hipEventRecord(L.stop, s);
  }
};

inline bool nonneg_finite(float v) { return v >= 0.0f && !isinf(v); }

#define TOPMOE_TRY(expr)                              \
  do {                                                \
    if ((expr) != hipSuccess) return TOPMOE_ERR_HIP;  \
  } while (0)

}  // namespace topmoe
