// scan_window_step.h -- sliding-window attention of one token a request over a
// ring of S + W cached keys: its arguments, and the bf16 kernel's calls.
#pragma once

#include "scan_mixer.h"

namespace scan {

struct WinStepArgs {
  scan_view4 q, k, v, o;
  void *kc, *vc;  // [n_slots, S + W, Hk, D]
  const int32_t* slots;
  const int32_t* pos;
  int64_t n_slots, cap;  // cap = S + W
  int64_t W, S;
  int Hq, Hk, D;
  float scale;
};

bool window_step_fits(const WinStepArgs& a, scan_dtype dt);
cudaError_t launch_window_step(const WinStepArgs& a, int64_t B, cudaStream_t s);

}  // namespace scan
