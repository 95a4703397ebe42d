// scan_mixer.h -- what the token-mixer operators around the scans share: the
// norm and rotation of queries and keys (scan_qknorm.cu), linear attention with
// a decay for each head (scan_linattn*.cu) and attention with a sliding window
// and first tokens that stay visible (scan_window*.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/libscan.h"
#include "scan_internal.h"

namespace scan {

constexpr int kMixMaxDim = 128;  // largest head dimension of the attention operators

// A [B, T, H, D] operand with unit stride along D; strides in elements.
template <typename T>
struct View {
  T* p;
  int64_t sb, st, sh;
  __host__ __device__ T* row(int64_t b, int64_t t, int64_t h) const {
    return p + b * sb + t * st + h * sh;
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Bounds of sequence i, forced into [0, T] whatever the device array holds, so
// that malformed offsets never lead out of the tensors.
__device__ __forceinline__ void seq_bounds(const int32_t* cu, int i, int64_t T, int64_t* beg,
                                           int64_t* end) {
  int64_t a = cu[i], e = cu[i + 1];
  a = a < 0 ? 0 : (a > T ? T : a);
  e = e < a ? a : (e > T ? T : e);
  *beg = a;
  *end = e;
}

// Records SCAN_ERR_SEQLENS unless 0 = cu[0] <= ... <= cu[n] = T. One warp.
__device__ __forceinline__ void check_seqlens(const int32_t* cu, int n, int64_t T, WsHeader* hdr) {
  bool bad = false;
  for (int i = threadIdx.x & 31; i <= n; i += 32) {
    const int64_t v = cu[i];
    if (i == 0 && v != 0) bad = true;
    if (i == n && v != T) bad = true;
    if (i < n && cu[i + 1] < v) bad = true;
  }
  if (bad && hdr) hdr->status = SCAN_ERR_SEQLENS;
}

// The sequence and the place in it of row tile `tile` when every sequence is
// cut into tiles of `rows` rows. One warp; false past the last tile.
__device__ __forceinline__ bool locate_tile(const int32_t* cu, int n, int64_t T, int64_t tile,
                                            int rows, int64_t* beg, int64_t* end, int64_t* local,
                                            int* seq = nullptr) {
  const int lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int base = 0; base < n; base += 32) {
    int64_t a = 0, e = 0;
    if (base + lane < n) seq_bounds(cu, base + lane, T, &a, &e);
    const int mine = (int)((e - a + rows - 1) / rows);
    int upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const bool here = tile >= before + upto - mine && tile < before + upto;
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int src = __ffs(who) - 1;
      *beg = __shfl_sync(0xffffffffu, a, src);
      *end = __shfl_sync(0xffffffffu, e, src);
      *local = tile - before - __shfl_sync(0xffffffffu, upto - mine, src);
      if (seq) *seq = base + src;
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

bool heads_map_fits(const scan_view4& v, int64_t B, int64_t T, int64_t H);
bool encode_heads_map(CUtensorMap* m, const scan_view4& v, int64_t B, int64_t T, int64_t H, int64_t D,
                      int rows);

// ---------------------------------------------------------------------------
// linear attention: one direction of the recurrence
//   S_t = lambda S_{t-1} + x2_t x3_t^T,  out_t = scale x1_t S_t       (forward)
//   S_t = x2_t x3_t^T + lambda S_{t+1},  out_t = scale x1_t S_t       (reverse)
// with S of K x V. The forward's initial state decays before the first step,
// the reverse's does not (it is the gradient of the state after the last
// step), and the reverse's final state is decayed once more (the gradient of
// the state before the first step). The forward pass is one such pass, the
// backward three: dq = (dout, v, k), dk = reverse (v, dout, q), dv = reverse
// (k, q, dout).
struct LinPass {
  scan_view4 x1, x2, x3, out;
  const float* s_in;   // nullable initial state of each (sequence, head)
  float* s_out;        // nullable final state
  int s_in_t;          // 1: s_in is stored V x K
  float s_in_mul;      // s_in is multiplied by this
  float s_out_mul;     // the final state by this
  int K, V;
  int reverse;
};

struct LinArgs {
  LinPass pass[3];
  int npass;
  const float* log_decay;  // [H]
  const int32_t* cu;
  int n_seqs;
  int64_t B, T;
  int H;
  float scale;
  WsHeader* hdr;
  float* ws;             // after the header
};

cudaError_t launch_linattn_general(const LinArgs& a, scan_dtype dt, cudaStream_t s);

// ---------------------------------------------------------------------------
// sliding-window attention
struct WinArgs {
  scan_view4 q, k, v, o, dout, dq, dk, dv;
  float* lse;    // [B, Hq, Tq]
  float* delta;  // [B, Hq, Tq] (workspace): sum of dout o
  const int32_t* cu;
  int n_seqs;
  int64_t B, Tq, Tk;
  int Hq, Hk, D;
  int64_t W, S;  // key j is seen by position i where j <= i and (i - j < W or j < S)
  float scale;
  WsHeader* hdr;
  float* ws;
};

// Tiles of `rows` keys that the queries at positions [p0, p1] see: those that hold
// first tokens, [0, sink), and those of the window, [near, last].
struct KeyTiles {
  int64_t sink, near, last;  // sink <= near; last < near: none
  __device__ int64_t count() const { return sink + (last >= near ? last - near + 1 : 0); }
  __device__ int64_t at(int64_t i) const { return i < sink ? i : near + (i - sink); }
};
__device__ __forceinline__ KeyTiles key_tiles(int64_t p0, int64_t p1, int64_t Tk, int64_t W, int64_t S,
                                              int rows) {
  KeyTiles t{0, 0, -1};
  if (p1 < 0 || Tk <= 0) return t;
  const int64_t hi = p1 < Tk ? p1 : Tk - 1;
  int64_t lo = p0 - W + 1;
  lo = lo < 0 ? 0 : lo;
  t.near = lo / rows;
  t.last = hi / rows;
  const int64_t s = S < hi + 1 ? S : hi + 1;
  const int64_t ns = (s + rows - 1) / rows;
  t.sink = ns < t.near ? ns : t.near;
  return t;
}

// Where a tile of rows lies: the sequence it belongs to and its first row there.
struct TileRows {
  int64_t qbeg, kbeg;   // first query and key row of the sequence
  int64_t nq, nk, off;  // rows of each, and the position of the first query
  int64_t t0;           // first row of the tile within the sequence
};
// Tile `tile` of `rows` rows; a whole warp (packed sequences are searched). False
// past the last tile.
__device__ __forceinline__ bool tile_rows(const int32_t* cu, int n_seqs, int64_t Tq, int64_t Tk,
                                          int64_t tile, int rows, TileRows* r) {
  if (!cu) {
    *r = TileRows{0, 0, Tq, Tk, Tk - Tq, tile * rows};
    return true;
  }
  int64_t beg, end, local;
  if (!locate_tile(cu, n_seqs, Tq, tile, rows, &beg, &end, &local)) return false;
  *r = TileRows{beg, beg, end - beg, end - beg, 0, local * rows};
  return true;
}

cudaError_t launch_window_general_fwd(const WinArgs& a, scan_dtype dt, cudaStream_t s);
cudaError_t launch_window_general_bwd(const WinArgs& a, scan_dtype dt, cudaStream_t s);

}  // namespace scan
