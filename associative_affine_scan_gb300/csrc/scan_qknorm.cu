// scan_qknorm.cu -- RMS norm of every query and key head with the position
// rotation in the same pass, forward and backward.
//
//   n = x r, r = (mean(x^2) + eps)^(-1/2),  z = w n,  y = rotate(z)
//   rotate: each pair (a, b) of the first R elements becomes
//           (a cos - b sin, a sin + b cos) with the cosine and sine of its
//           position and frequency; elements R.. are left as they are
//   backward: dz = rotate by the opposite angle (dy), g = w dz,
//             dx = r (g - n mean(g n)),  dw = sum over rows of dz n
//
// Bound by DRAM: one read and one write of every element forward, two reads
// and one write backward, about ten operations on each. A row of D elements is
// held by the 8, 16 or 32 lanes that cover it, eight elements a lane, so the
// norm's sum is three to five shuffles and no row is read twice. A lane's eight
// elements are four pairs (elements 4u.. and R/2 + 4u.., or 8u.. where
// neighbours are paired), so the rotation needs no exchange. A group of lanes
// takes up to four heads of one token: the token's cosines and sines are read
// once for them, and four rows are in flight a lane.
#include "scan_mixer.h"

namespace scan {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;  // heads of one token that a group of lanes takes

struct QkArgs {
  scan_view4 x[2], y[2], dy[2], dx[2];  // queries, keys
  const float* w[2];                    // nullable (ones)
  const float* cs;
  const float* sn;
  const int32_t* pos;
  float* part;   // backward: [blocks][2][D] partial weight gradients
  float* dw[2];
  int64_t BT, T, P;
  int H[2];
  int chunks[2];  // ceil(H / kHeads)
  int D, R;
  int pairs;
  float eps;
};

// Eight elements of a row: two runs of four (rotated halves apart) or one of eight.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int lo, int hi, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* row, int lo, int hi, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(row + lo);
  const float4 b = *reinterpret_cast<const float4*>(row + hi);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* row, int lo, int hi,
                                                     float (&v)[8]) {
  const uint2 a = *reinterpret_cast<const uint2*>(row + lo);
  const uint2 b = *reinterpret_cast<const uint2*>(row + hi);
  const uint32_t u[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* row, int lo, int hi, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<float>(float* row, int lo, int hi, const float (&v)[8]) {
  *reinterpret_cast<float4*>(row + lo) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(row + hi) = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* row, int lo, int hi,
                                                      const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint2*>(row + lo) = make_uint2(u[0], u[1]);
  *reinterpret_cast<uint2*>(row + hi) = make_uint2(u[2], u[3]);
}

// What a lane holds of a row, and the cosines and sines of its pairs.
struct Unit {
  int lo, hi;   // elements lo..lo+3 and hi..hi+3
  int rot;      // its pairs are rotated
  int cs;       // first of its four table entries
  bool on;      // the lane holds part of the row
};

__device__ __forceinline__ Unit unit_of(int u, const QkArgs& a) {
  Unit t;
  t.on = 8 * u < a.D;
  t.rot = 8 * u < a.R;
  t.cs = 4 * u;
  if (t.rot && !a.pairs) {
    t.lo = 4 * u;
    t.hi = a.R / 2 + 4 * u;
  } else {
    t.lo = 8 * u;
    t.hi = 8 * u + 4;
  }
  return t;
}

// (a, b) -> (a c - b s, a s + b c) on a lane's four pairs.
__device__ __forceinline__ void rotate(float (&v)[8], const float (&c)[4], const float (&s)[4],
                                       bool pairs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = pairs ? 2 * i : i, ib = pairs ? 2 * i + 1 : 4 + i;
    const float x = v[ia], y = v[ib];
    v[ia] = x * c[i] - y * s[i];
    v[ib] = x * s[i] + y * c[i];
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = G / 2; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// The token's cosines and sines; a position outside the tables gives NaN, so
// that the mistake shows in the result instead of reading past them.
__device__ __forceinline__ void load_turn(const QkArgs& a, int64_t tok, const Unit& u, float (&c)[4],
                                          float (&s)[4]) {
  const int64_t p = a.pos ? (int64_t)a.pos[tok] : tok % a.T;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
  if (!u.rot) return;
  if (p < 0 || p >= a.P) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
    return;
  }
  const float4 cv = *reinterpret_cast<const float4*>(a.cs + p * (a.R / 2) + u.cs);
  const float4 sv = *reinterpret_cast<const float4*>(a.sn + p * (a.R / 2) + u.cs);
  c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
  s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
}

__device__ __forceinline__ void load_weight(const float* w, const Unit& u, float (&v)[8]) {
  if (w && u.on) load8<float>(w, u.lo, u.hi, v);
  else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  }
}

template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qknorm_fwd_kernel(const QkArgs a) {
  const int per = a.chunks[0] + a.chunks[1];
  const int64_t item = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G;
  const bool live = item < a.BT * per;  // lanes of a dead group stay for the shuffles
  const int64_t tok = live ? item / per : 0;
  int c = live ? (int)(item % per) : 0;
  const int m = c >= a.chunks[0];
  if (m) c -= a.chunks[0];
  const Unit u = unit_of(threadIdx.x % G, a);
  const int64_t b = tok / a.T, t = tok % a.T;
  const int h0 = c * kHeads;
  const View<const T> x = {static_cast<const T*>(a.x[m].ptr), a.x[m].stride_b, a.x[m].stride_t,
                           a.x[m].stride_h};
  const View<T> y = {static_cast<T*>(a.y[m].ptr), a.y[m].stride_b, a.y[m].stride_t, a.y[m].stride_h};
  float v[kHeads][8];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (live && u.on && h0 + i < a.H[m]) load8<T>(x.row(b, t, h0 + i), u.lo, u.hi, v[i]);
  }
  float cs[4], sn[4], w[8];
  load_turn(a, tok, u, cs, sn);
  load_weight(a.w[m], u, w);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sq = fmaf(v[i][j], v[i][j], sq);
    const float r = rsqrtf(group_sum<G>(sq) / (float)a.D + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] *= r * w[j];
    if (u.rot) rotate(v[i], cs, sn, PAIRS);
    if (live && u.on && h0 + i < a.H[m]) store8<T>(y.row(b, t, h0 + i), u.lo, u.hi, v[i]);
  }
}

// Each block walks tokens with the weight gradients in registers and leaves one
// partial sum; the partial sums are added in block order by the kernel below,
// so the result does not depend on the order in which blocks finish.
template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qknorm_bwd_kernel(const QkArgs a) {
  const int per = a.chunks[0] + a.chunks[1];
  const int ng = kThreads / G;
  const Unit u = unit_of(threadIdx.x % G, a);
  float dw[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.f;
  const int64_t total = a.BT * per;
  const int64_t step = (int64_t)gridDim.x * ng;
  // whole warps leave together: the bound is on the warp's first group
  for (int64_t base = (int64_t)blockIdx.x * ng + (threadIdx.x / 32) * (32 / G); base < total;
       base += step) {
    const int64_t item = base + (threadIdx.x % 32) / G;
    const bool live = item < total;
    const int64_t tok = live ? item / per : 0;
    int c = live ? (int)(item % per) : 0;
    const int m = c >= a.chunks[0];
    if (m) c -= a.chunks[0];
    const int64_t b = tok / a.T, t = tok % a.T;
    const int h0 = c * kHeads;
    const View<const T> x = {static_cast<const T*>(a.x[m].ptr), a.x[m].stride_b, a.x[m].stride_t,
                             a.x[m].stride_h};
    const View<const T> dy = {static_cast<const T*>(a.dy[m].ptr), a.dy[m].stride_b,
                              a.dy[m].stride_t, a.dy[m].stride_h};
    const View<T> dx = {static_cast<T*>(a.dx[m].ptr), a.dx[m].stride_b, a.dx[m].stride_t,
                        a.dx[m].stride_h};
    float v[kHeads][8], g[kHeads][8];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = g[i][j] = 0.f;
      if (live && u.on && h0 + i < a.H[m]) {
        load8<T>(x.row(b, t, h0 + i), u.lo, u.hi, v[i]);
        load8<T>(dy.row(b, t, h0 + i), u.lo, u.hi, g[i]);
      }
    }
    float cs[4], sn[4], w[8];
    load_turn(a, tok, u, cs, sn);
    load_weight(a.w[m], u, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) sn[i] = -sn[i];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const bool here = live && u.on && h0 + i < a.H[m];
      if (u.rot) rotate(g[i], cs, sn, PAIRS);
      float sq = 0.f, gn = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sq = fmaf(v[i][j], v[i][j], sq);
        gn = fmaf(g[i][j] * w[j], v[i][j], gn);
      }
      const float r = rsqrtf(group_sum<G>(sq) / (float)a.D + a.eps);
      const float mean = group_sum<G>(gn) * r / (float)a.D;  // mean(g n)
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[i][j] * r;
        const float d = here ? g[i][j] * n : 0.f;
        if (m) dw[1][j] += d;
        else dw[0][j] += d;
        o[j] = r * (g[i][j] * w[j] - n * mean);
      }
      if (here) store8<T>(dx.row(b, t, h0 + i), u.lo, u.hi, o);
    }
  }
  // groups of the block, in order
  __shared__ float red[kThreads * 8];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[threadIdx.x * 8 + j] = dw[m][j];
    __syncthreads();
    if (threadIdx.x < G && u.on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float s = 0.f;
        for (int k = 0; k < ng; ++k) s += red[(k * G + threadIdx.x) * 8 + j];
        a.part[((int64_t)blockIdx.x * 2 + m) * a.D + (j < 4 ? u.lo + j : u.hi + j - 4)] = s;
      }
    }
  }
}

// Columns of the partial sums, one block per (matrix, 32 columns): 32 lanes of
// columns by eight slices of blocks, the slices then added in order.
__global__ void __launch_bounds__(256) qknorm_dw_kernel(const QkArgs a, int blocks) {
  const int m = blockIdx.y, col = blockIdx.x * 32 + threadIdx.x % 32, sl = threadIdx.x / 32;
  __shared__ float red[8][32];
  float s = 0.f;
  if (col < a.D)
    for (int k = sl; k < blocks; k += 8) s += a.part[((int64_t)k * 2 + m) * a.D + col];
  red[sl][threadIdx.x % 32] = s;
  __syncthreads();
  if (sl == 0 && col < a.D && a.dw[m]) {
    for (int k = 1; k < 8; ++k) s += red[k][threadIdx.x % 32];
    a.dw[m][col] = s;
  }
}

constexpr int kBwdBlocks = 152 * 4;

int group_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

template <typename T, int G>
cudaError_t qk_launch_g(const QkArgs& a, bool fwd, cudaStream_t s) {
  const int64_t items = a.BT * (a.chunks[0] + a.chunks[1]);
  const int64_t need = (items + kThreads / G - 1) / (kThreads / G);
  if (fwd) {
    if (a.pairs) qknorm_fwd_kernel<T, G, true><<<(unsigned)need, kThreads, 0, s>>>(a);
    else qknorm_fwd_kernel<T, G, false><<<(unsigned)need, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const int blocks = (int)(need < kBwdBlocks ? need : kBwdBlocks);
  if (a.pairs) qknorm_bwd_kernel<T, G, true><<<blocks, kThreads, 0, s>>>(a);
  else qknorm_bwd_kernel<T, G, false><<<blocks, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  qknorm_dw_kernel<<<dim3((a.D + 31) / 32, 2), 256, 0, s>>>(a, blocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t qk_launch(const QkArgs& a, bool fwd, cudaStream_t s) {
  switch (group_lanes(a.D)) {
    case 8: return qk_launch_g<T, 8>(a, fwd, s);
    case 16: return qk_launch_g<T, 16>(a, fwd, s);
    default: return qk_launch_g<T, 32>(a, fwd, s);
  }
}

bool view_aligned(const scan_view4* v, scan_dtype dt) {
  const int64_t n = dt == SCAN_BF16 ? 8 : 4;  // elements of 16 bytes
  return (uintptr_t)v->ptr % 16 == 0 && v->stride_b % n == 0 && v->stride_t % n == 0 &&
         v->stride_h % n == 0;
}

scan_status qk_args(QkArgs* a, const scan_view4* q, const scan_view4* k, const float* qw,
                    const float* kw, const float* cs, const float* sn, const int32_t* pos, int64_t B,
                    int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t P,
                    int32_t interleaved, float eps, scan_dtype dt) {
  if (dt != SCAN_F32 && dt != SCAN_BF16) return SCAN_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || Hq < 0 || Hk < 0 || D < 1 || R < 0 || R > D || P < 0)
    return SCAN_ERR_INVALID_ARG;
  if (!(eps >= 0.f)) return SCAN_ERR_INVALID_ARG;
  if (D % 8 || D > 256 || R % 8) return SCAN_ERR_UNSUPPORTED;
  if (Hq > (1 << 20) || Hk > (1 << 20)) return SCAN_ERR_UNSUPPORTED;
  // grid.x counts blocks of at least 8 items; the product is bounded step by step
  if (B > (1LL << 31) || T > (1LL << 31) || B * T > (1LL << 40)) return SCAN_ERR_UNSUPPORTED;
  if (B * T * ((Hq + 3) / 4 + (Hk + 3) / 4) / 8 >= 0x7fffffffLL) return SCAN_ERR_UNSUPPORTED;
  if (R > 0 && B * T > 0 && (!cs || !sn)) return SCAN_ERR_INVALID_ARG;
  if ((uintptr_t)cs % 16 || (uintptr_t)sn % 16 || (uintptr_t)qw % 16 || (uintptr_t)kw % 16)
    return SCAN_ERR_ALIGNMENT;
  const bool some = B * T > 0;  // an empty tensor may have no address
  if ((Hq && (!q || (some && !q->ptr))) || (Hk && (!k || (some && !k->ptr)))) return SCAN_ERR_INVALID_ARG;
  *a = QkArgs{};
  if (Hq) a->x[0] = *q;
  if (Hk) a->x[1] = *k;
  a->w[0] = qw;
  a->w[1] = kw;
  a->cs = cs;
  a->sn = sn;
  a->pos = pos;
  a->BT = B * T;
  a->T = T > 0 ? T : 1;
  a->P = P;
  a->H[0] = (int)Hq;
  a->H[1] = (int)Hk;
  a->chunks[0] = (int)((Hq + kHeads - 1) / kHeads);
  a->chunks[1] = (int)((Hk + kHeads - 1) / kHeads);
  a->D = (int)D;
  a->R = (int)R;
  a->pairs = interleaved != 0;
  a->eps = eps;
  for (int m = 0; m < 2; ++m)
    if (a->H[m] && !view_aligned(&a->x[m], dt)) return SCAN_ERR_ALIGNMENT;
  return SCAN_OK;
}

}  // namespace
}  // namespace scan

using namespace scan;

extern "C" {

size_t qk_norm_rope_workspace_bytes(int64_t D) {
  if (D < 1 || D % 8 || D > 256) return 0;
  return (size_t)kBwdBlocks * 2 * (size_t)D * 4;
}

scan_status qk_norm_rope_fwd(const scan_view4* q, const scan_view4* k, const float* q_weight,
                             const float* k_weight, const float* cos_table, const float* sin_table,
                             const int32_t* positions, const scan_view4* q_out,
                             const scan_view4* k_out, int64_t B, int64_t T, int64_t Hq, int64_t Hk,
                             int64_t D, int64_t R, int64_t P, int32_t interleaved, float eps,
                             scan_dtype dt, cudaStream_t stream) {
  QkArgs a;
  const scan_status st = qk_args(&a, q, k, q_weight, k_weight, cos_table, sin_table, positions, B, T,
                                 Hq, Hk, D, R, P, interleaved, eps, dt);
  if (st != SCAN_OK) return st;
  if (a.BT * (Hq + Hk) == 0) return SCAN_OK;
  if ((Hq && (!q_out || !q_out->ptr)) || (Hk && (!k_out || !k_out->ptr))) return SCAN_ERR_INVALID_ARG;
  if (Hq) a.y[0] = *q_out;
  if (Hk) a.y[1] = *k_out;
  for (int m = 0; m < 2; ++m)
    if (a.H[m] && !view_aligned(&a.y[m], dt)) return SCAN_ERR_ALIGNMENT;
  const cudaError_t e = dt == SCAN_BF16 ? qk_launch<__nv_bfloat16>(a, true, stream)
                                        : qk_launch<float>(a, true, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status qk_norm_rope_bwd(const scan_view4* q, const scan_view4* k, const float* q_weight,
                             const float* k_weight, const float* cos_table, const float* sin_table,
                             const int32_t* positions, const scan_view4* dq_out,
                             const scan_view4* dk_out, const scan_view4* dq, const scan_view4* dk,
                             float* dq_weight, float* dk_weight, int64_t B, int64_t T, int64_t Hq,
                             int64_t Hk, int64_t D, int64_t R, int64_t P, int32_t interleaved,
                             float eps, scan_dtype dt, void* workspace, size_t workspace_bytes,
                             cudaStream_t stream) {
  QkArgs a;
  const scan_status st = qk_args(&a, q, k, q_weight, k_weight, cos_table, sin_table, positions, B, T,
                                 Hq, Hk, D, R, P, interleaved, eps, dt);
  if (st != SCAN_OK) return st;
  a.dw[0] = dq_weight;
  a.dw[1] = dk_weight;
  if (a.BT * (Hq + Hk) == 0) {  // no rows: the weight gradients are 0
    cudaError_t e = cudaSuccess;
    if (dq_weight) e = launch_fill_zero(dq_weight, D, stream);
    if (e == cudaSuccess && dk_weight) e = launch_fill_zero(dk_weight, D, stream);
    return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
  }
  const scan_view4* in[2] = {dq_out, dk_out};
  const scan_view4* out[2] = {dq, dk};
  for (int m = 0; m < 2; ++m) {
    if (!a.H[m]) continue;
    if (!in[m] || !in[m]->ptr || !out[m] || !out[m]->ptr) return SCAN_ERR_INVALID_ARG;
    if (!view_aligned(in[m], dt) || !view_aligned(out[m], dt)) return SCAN_ERR_ALIGNMENT;
    a.dy[m] = *in[m];
    a.dx[m] = *out[m];
  }
  if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < qk_norm_rope_workspace_bytes(D))
    return SCAN_ERR_WORKSPACE;
  a.part = static_cast<float*>(workspace);
  const cudaError_t e = dt == SCAN_BF16 ? qk_launch<__nv_bfloat16>(a, false, stream)
                                        : qk_launch<float>(a, false, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // extern "C"
