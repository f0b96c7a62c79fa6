// Helpers of the C ABI's host side.
#pragma once

#include <cstddef>
#include <cstdint>

#include "kda_internal.h"

namespace kda {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

inline kda_status_t hip_status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

// Records the caller's timing event `which` (0 = before, 1 = after) of a stage.
inline void mark(const kda_config_t* cfg, int stage, int which, hipStream_t st) {
  if (!cfg->stage_events) return;
  void* ev = cfg->stage_events[2 * stage + which];
  if (ev) (void)hipEventRecord(static_cast<hipEvent_t>(ev), st);
}

// Runs one stage's launcher between its two timing marks.
template <class F>
kda_status_t stage(const kda_config_t* cfg, int s, hipStream_t st, F&& launch) {
  mark(cfg, s, 0, st);
  const hipError_t e = launch();
  mark(cfg, s, 1, st);
  return hip_status(e);
}

}  // namespace kda
