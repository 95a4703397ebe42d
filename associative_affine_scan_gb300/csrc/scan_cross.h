// scan_cross.h -- attention to the states of another sequence (an encoder's): its
// arguments, and which of its kernels takes a call.
#pragma once

#include "scan_mixer.h"

namespace scan {

// Whole rows: batch row b's queries see the first lens[b] keys of row b (all Tk
// without lens). Packed (cu_q): sequence i's queries see sequence i's keys.
struct CrossArgs {
  scan_view4 q, k, v, o, dout, dq, dk, dv;
  float* lse;           // [B, Hq, Tq]
  float* delta;         // [B, Hq, Tq] (workspace): sum of dout o
  const int32_t* lens;  // [B], nullable
  const int32_t* cu_q;  // [n_seqs + 1], nullable
  const int32_t* cu_k;
  int n_seqs;
  int64_t B, Tq, Tk;
  int Hq, Hk, D;
  float scale;
  WsHeader* hdr;
  float* ws;  // after delta
};

// Keys that batch row b has, forced into [0, Tk] whatever the array holds.
__device__ __forceinline__ int64_t keys_of(const int32_t* lens, int64_t b, int64_t Tk) {
  if (!lens) return Tk;
  const int64_t n = lens[b];
  return n < 0 ? 0 : n > Tk ? Tk : n;
}

// Where a tile of rows lies: first query and key row of its sequence, rows of each,
// and the tile's first row within the sequence.
struct CrossRows {
  int64_t qbeg, kbeg, nq, nk, t0;
};
// Tile `tile` of `rows` query rows (by_keys: key rows) of batch row b; a whole warp
// (packed sequences are searched). False past the last tile.
__device__ __forceinline__ bool cross_rows(const int32_t* lens, const int32_t* cu_q, const int32_t* cu_k, int n_seqs,
                                           int64_t Tq, int64_t Tk, int64_t b, int64_t tile, int rows, bool by_keys,
                                           CrossRows* r) {
  if (!cu_q) {
    *r = CrossRows{0, 0, Tq, keys_of(lens, b, Tk), tile * rows};
    return true;
  }
  int64_t beg, end, local, obeg, oend;
  int seq;
  if (!locate_tile(by_keys ? cu_k : cu_q, n_seqs, by_keys ? Tk : Tq, tile, rows, &beg, &end, &local, &seq)) return false;
  seq_bounds(by_keys ? cu_q : cu_k, seq, by_keys ? Tq : Tk, &obeg, &oend);
  *r = by_keys ? CrossRows{obeg, beg, oend - obeg, end - beg, local * rows}
               : CrossRows{beg, obeg, end - beg, oend - obeg, local * rows};
  return true;
}
// Sequences (batch rows) whose keys are of many numbers are worked on from the longest to
// the shortest, where a warp can look them all over; a table in shared memory says which
// sequence the i-th tile is of. And blocks go through the tiles forth and back, item_of, so
// that who had the longest of one round has the shortest of the next (seven packed sequences,
// 12 heads of 96, forward and backward of 4001 queries over 5003 keys in us: 165 in the
// order of the sequences, 153 so).
struct Order {
  int64_t start[32];  // the sequence's first tile; by the numbers of keys
  int tiles[32], seq[32];
  // A warp. units: tiles that differ in their heads only.
  __device__ __forceinline__ void make(const int32_t* lens, const int32_t* cu_q, const int32_t* cu_k, int n_seqs,
                                       int64_t B, int64_t Tq, int64_t Tk, int rows, int64_t units) {
    const int lane = threadIdx.x & 31, n = cu_q ? n_seqs : (int)B;
    int keys = -1, mine = 0;
    if (lane < n) {
      int64_t qa = 0, qe = Tq, ka = 0, ke = 0;
      if (cu_q) {
        seq_bounds(cu_q, lane, Tq, &qa, &qe);
        seq_bounds(cu_k, lane, Tk, &ka, &ke);
      } else {
        ke = keys_of(lens, lane, Tk);
      }
      keys = (int)(ke - ka);
      mine = (int)((qe - qa + rows - 1) / rows);
    }
    int rank = 0;
    int64_t before = 0;
    for (int i = 0; i < 32; ++i) {
      const int k = __shfl_sync(0xffffffffu, keys, i), t = __shfl_sync(0xffffffffu, mine, i);
      if (k > keys || (k == keys && i < lane)) {
        ++rank;
        before += t;
      }
    }
    start[rank] = before * units;
    tiles[rank] = mine;
    seq[rank] = lane;
  }
  // Sequence, unit and tile of item i; false past the last. A warp.
  __device__ __forceinline__ bool find(int64_t i, int64_t units, int* s, int64_t* unit, int64_t* tile) const {
    const int at = 31 - __clz(__ballot_sync(0xffffffffu, i >= start[threadIdx.x & 31]));
    const int64_t t = tiles[at], n = i - start[at];
    if (t == 0 || n >= t * units) return false;
    *s = seq[at];
    *unit = n / t;
    *tile = n - *unit * t;
    return true;
  }
};
__host__ __device__ inline bool orders(const int32_t* lens, const int32_t* cu_q, int n_seqs, int64_t B) {
  return (cu_q ? n_seqs : lens ? B : 33) <= 32;
}
__device__ __forceinline__ int64_t item_of(int64_t round, int order) {
  return round * gridDim.x + (order && (round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
// The rows of tile `tile` of sequence (batch row) s.
__device__ __forceinline__ CrossRows rows_of(const int32_t* lens, const int32_t* cu_q, const int32_t* cu_k, int64_t Tq,
                                             int64_t Tk, int s, int64_t t0) {
  if (!cu_q) return CrossRows{0, 0, Tq, keys_of(lens, s, Tk), t0};
  int64_t qa, qe, ka, ke;
  seq_bounds(cu_q, s, Tq, &qa, &qe);
  seq_bounds(cu_k, s, Tk, &ka, &ke);
  return CrossRows{qa, ka, qe - qa, ke - ka, t0};
}

// Records malformed offsets or lengths. One warp.
__device__ __forceinline__ void check_cross(const int32_t* lens, const int32_t* cu_q, const int32_t* cu_k, int n_seqs,
                                            int64_t B, int64_t Tq, int64_t Tk, WsHeader* hdr) {
  if (cu_q) {
    check_seqlens(cu_q, n_seqs, Tq, hdr);
    check_seqlens(cu_k, n_seqs, Tk, hdr);
  } else if (lens) {
    bool bad = false;
    for (int64_t i = threadIdx.x & 31; i < B; i += 32) bad |= lens[i] < 0 || lens[i] > Tk;
    if (bad) hdr->status = SCAN_ERR_SEQLENS;
  }
}

// A kernel that is launched while the one before it runs, whose end it waits for itself.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_cross_general_fwd(const CrossArgs& a, scan_dtype dt, cudaStream_t s);
cudaError_t launch_cross_general_bwd(const CrossArgs& a, scan_dtype dt, cudaStream_t s);

// One query token a request over a pool of cached keys and values [n_slots, Tk, Hk, D].
struct CrossStepArgs {
  scan_view4 q, k, v, o;
  const int32_t* lens;   // [n_slots], nullable
  const int32_t* slots;  // [B], nullable
  int64_t n_slots, Tk;
  int Hq, Hk, D;
  float scale;
  WsHeader* hdr;
  void* ws;  // after the header
};

}  // namespace scan
