// scan_cross_tc.h -- the tensor-core form of attention to another sequence
// (scan_cross_fwd.cu, scan_cross_bwd.cu) and its form for single tokens
// (scan_cross_step.cu): which calls they take and their launches.
#pragma once

#include "scan_cross.h"

namespace scan {

bool cross_tc_fits(const CrossArgs& a, scan_dtype dt, bool backward);
cudaError_t launch_cross_tc_fwd(const CrossArgs& a, cudaStream_t s);

// Floats of workspace for the parts of the keys' tiles that blocks share.
size_t cross_tc_bwd_floats(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t D, int64_t n_seqs);
cudaError_t launch_cross_tc_bwd(const CrossArgs& a, cudaStream_t s);

// Bytes of workspace for the parts of the units that blocks share.
size_t cross_step_bytes(int64_t B, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D);
bool cross_step_fits(const CrossStepArgs& a, scan_dtype dt, int64_t B);
cudaError_t launch_cross_step(const CrossStepArgs& a, int64_t B, cudaStream_t s);

// Whether the rows of a [B, T, H, D] bf16 output start on 32 bytes and are whole pieces of them.
inline bool rows_on_32(const scan_view4& v, int64_t B, int64_t T, int64_t H, int64_t D) {
  return D % 16 == 0 && (uintptr_t)v.ptr % 32 == 0 && (B == 1 || v.stride_b % 16 == 0) &&
         (T == 1 || v.stride_t % 16 == 0) && (H == 1 || v.stride_h % 16 == 0);
}

}  // namespace scan
