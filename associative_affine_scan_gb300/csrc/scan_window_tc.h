// scan_window_tc.h -- the tensor-core form of sliding-window attention
// (scan_window_fwd.cu, scan_window_bwd.cu): which calls it takes and its launches.
#pragma once

#include "scan_mixer.h"

namespace scan {

bool window_tc_fits(const WinArgs& a, scan_dtype dt, bool backward);
cudaError_t launch_window_tc_fwd(const WinArgs& a, cudaStream_t s);

// Floats of workspace for the partial sums of the backward's cut key tiles.
size_t window_tc_bwd_floats(int64_t B, int64_t Tq, int64_t Tk, int64_t Hk, int64_t D, int64_t W, int64_t S,
                            bool packed);
cudaError_t launch_window_tc_bwd(const WinArgs& a, float* part, cudaStream_t s);

}  // namespace scan
