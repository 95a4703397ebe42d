// scan_cross_tc.h -- the tensor-core form of attention to another sequence
// (scan_cross_fwd.cu): which calls it takes and its launch.
#pragma once

#include "scan_cross.h"

namespace scan {

bool cross_tc_fits(const CrossArgs& a, scan_dtype dt, bool backward);
cudaError_t launch_cross_tc_fwd(const CrossArgs& a, cudaStream_t s);

}  // namespace scan
