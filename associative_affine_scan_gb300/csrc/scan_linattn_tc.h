// scan_linattn_tc.h -- the chunked tensor-core form of linear attention
// (scan_linattn_tc.cu): which calls it takes, its workspace and its launch.
#pragma once

#include "scan_mixer.h"

namespace scan {

bool linattn_tc_fits(const LinArgs& a, scan_dtype dt);
size_t linattn_tc_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                                  int64_t n_seqs);
cudaError_t launch_linattn_tc(const LinArgs& a, cudaStream_t s);

}  // namespace scan
