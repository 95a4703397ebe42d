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
// takes up to four heads of one token (two in the backward): the token's cosines
// and sines are read once for them. Blocks walk the tokens of either the queries
// or the keys, so that a lane keeps its weights (and sums of weight gradients) in
// registers, and read the next heads, their table entries and the position after
// that while they work on the current ones.
#include "scan_mixer.h"

namespace scan {
namespace {

constexpr int kThreads = 256;
constexpr int kFwdHeads = 4;  // heads of one token that a group of lanes takes
constexpr int kBwdHeads = 2;

struct QkArgs {
  scan_view4 x[2], y[2], dy[2], dx[2];  // queries, keys
  const float* w[2];                    // nullable (ones)
  const float* cs;
  const float* sn;
  const int32_t* pos;
  float* part;   // backward: [blocks][D] partial weight gradients, the queries' first
  float* dw[2];
  int64_t BT, T, P;
  int H[2];
  int chunks[2];  // groups of heads
  int blocks[2];  // blocks that walk the queries, and the keys
  int D, R;
  int pairs;
  float eps;
};

// Eight elements of a row as they are in memory: two runs of four (the halves of
// rotated pairs) or one of eight.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* row, int lo, int hi) {
    a = *reinterpret_cast<const float4*>(row + lo);
    b = *reinterpret_cast<const float4*>(row + hi);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int lo, int hi) {
    a = *reinterpret_cast<const uint2*>(row + lo);
    b = *reinterpret_cast<const uint2*>(row + hi);
  }
  __device__ __forceinline__ void clear() { a = b = make_uint2(0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
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

// Cosines and sines of position p; one outside the tables gives NaN, so that the
// mistake shows in the result instead of reading past them.
__device__ __forceinline__ void load_turn(const QkArgs& a, int64_t p, const Unit& u, float (&c)[4],
                                          float (&s)[4]) {
  if (!u.rot) return;
  const bool ok = p >= 0 && p < a.P;
  const int64_t at = (ok ? p : 0) * (a.R / 2) + u.cs;
  const float4 cv = *reinterpret_cast<const float4*>(a.cs + at);
  const float4 sv = *reinterpret_cast<const float4*>(a.sn + at);
  const float bad = __int_as_float(0x7fc00000);
  c[0] = ok ? cv.x : bad; c[1] = ok ? cv.y : bad; c[2] = ok ? cv.z : bad; c[3] = ok ? cv.w : bad;
  s[0] = ok ? sv.x : bad; s[1] = ok ? sv.y : bad; s[2] = ok ? sv.z : bad; s[3] = ok ? sv.w : bad;
}

__device__ __forceinline__ void load_weight(const float* w, const Unit& u, float (&v)[8]) {
  Raw<float> r;
  if (w && u.on) {
    r.load(w, u.lo, u.hi);
    r.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  }
}

// A group's place in its walk over (token, heads): items `step` apart.
struct Walk {
  int64_t item, b, t;
  int c;
  int64_t step, db, dt;
  int dc;
  __device__ __forceinline__ Walk(const QkArgs& a, int m, int64_t first, int64_t by) {
    const int per = a.chunks[m];
    item = first;
    step = by;
    c = (int)(first % per);
    const int64_t tok = first / per;
    b = tok / a.T;
    t = tok % a.T;
    dc = (int)(by % per);
    const int64_t dtok = by / per;
    db = dtok / a.T;
    dt = dtok % a.T;
  }
  __device__ __forceinline__ void next(const QkArgs& a, int m) {
    item += step;
    b += db;
    t += dt;
    c += dc;
    if (c >= a.chunks[m]) c -= a.chunks[m], ++t;
    if (t >= a.T) t -= a.T, ++b;
  }
  __device__ __forceinline__ int64_t position(const QkArgs& a) const {
    return a.pos ? (int64_t)a.pos[b * a.T + t] : t;
  }
};

template <typename T, int N>
__device__ __forceinline__ void load_heads(const View<const T>& x, const Walk& w, const Unit& u, int H, bool live,
                                           Raw<T> (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (live && u.on && w.c * N + i < H) r[i].load(x.row(w.b, w.t, w.c * N + i), u.lo, u.hi);
    else r[i].clear();
  }
}

template <typename T>
__device__ __forceinline__ View<T> qk_view(const scan_view4& v) {
  return View<T>{static_cast<T*>(v.ptr), v.stride_b, v.stride_t, v.stride_h};
}

template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qknorm_fwd_kernel(const QkArgs a) {
  constexpr int N = kFwdHeads;
  const int m = blockIdx.x >= a.blocks[0];
  const int64_t block = m ? blockIdx.x - a.blocks[0] : blockIdx.x;
  const int64_t items = a.BT * a.chunks[m];
  const Unit u = unit_of(threadIdx.x % G, a);
  const View<const T> x = m ? qk_view<const T>(a.x[1]) : qk_view<const T>(a.x[0]);
  const View<T> y = m ? qk_view<T>(a.y[1]) : qk_view<T>(a.y[0]);
  const int H = a.H[m];
  Walk w(a, m, block * (kThreads / G) + threadIdx.x / G, (int64_t)a.blocks[m] * (kThreads / G));
  Walk ahead = w;
  float wt[8], cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  Raw<T> r[N];
  load_heads<T, N>(x, w, u, H, w.item < items, r);
  if (w.item < items) load_turn(a, w.position(a), u, cs, sn);
  load_weight(a.w[m], u, wt);
  ahead.next(a, m);
  int64_t p1 = ahead.item < items ? ahead.position(a) : 0;
  // whole warps leave together: the bound is on the warp's first group
  int64_t lead = w.item - (threadIdx.x % 32) / G;
  while (lead < items) {
    const bool more = ahead.item < items;
    Raw<T> r1[N];
    float cs1[4] = {1.f, 1.f, 1.f, 1.f}, sn1[4] = {0.f, 0.f, 0.f, 0.f};
    load_heads<T, N>(x, ahead, u, H, more, r1);
    if (more) load_turn(a, p1, u, cs1, sn1);
    const Walk now = w;
    w = ahead;
    ahead.next(a, m);
    if (ahead.item < items) p1 = ahead.position(a);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float v[8], sq = 0.f;
      r[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) sq = fmaf(v[j], v[j], sq);
      const float rs = rsqrtf(group_sum<G>(sq) / (float)a.D + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= rs * wt[j];
      if (u.rot) rotate(v, cs, sn, PAIRS);
      if (now.item < items && u.on && now.c * N + i < H)
        store8<T>(y.row(now.b, now.t, now.c * N + i), u.lo, u.hi, v);
      r[i] = r1[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = cs1[i], sn[i] = sn1[i];
    lead += w.step;
  }
}

// Each block leaves one partial sum of its weight's gradient; the partial sums are
// added in block order by the kernel below, so the result does not depend on the
// order in which blocks finish.
template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qknorm_bwd_kernel(const QkArgs a) {
  constexpr int N = kBwdHeads, NG = kThreads / G;
  const int m = blockIdx.x >= a.blocks[0];
  const int64_t block = m ? blockIdx.x - a.blocks[0] : blockIdx.x;
  const int64_t items = a.BT * a.chunks[m];
  const Unit u = unit_of(threadIdx.x % G, a);
  const View<const T> x = m ? qk_view<const T>(a.x[1]) : qk_view<const T>(a.x[0]);
  const View<const T> dy = m ? qk_view<const T>(a.dy[1]) : qk_view<const T>(a.dy[0]);
  const View<T> dx = m ? qk_view<T>(a.dx[1]) : qk_view<T>(a.dx[0]);
  const int H = a.H[m];
  Walk w(a, m, block * NG + threadIdx.x / G, (int64_t)a.blocks[m] * NG);
  Walk ahead = w;
  float wt[8], dw[8], cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = 0.f;
  Raw<T> r[N], g[N];
  load_heads<T, N>(x, w, u, H, w.item < items, r);
  load_heads<T, N>(dy, w, u, H, w.item < items, g);
  if (w.item < items) load_turn(a, w.position(a), u, cs, sn);
  load_weight(a.w[m], u, wt);
  ahead.next(a, m);
  int64_t p1 = ahead.item < items ? ahead.position(a) : 0;
  int64_t lead = w.item - (threadIdx.x % 32) / G;
  while (lead < items) {
    const bool more = ahead.item < items;
    Raw<T> r1[N], g1[N];
    float cs1[4] = {1.f, 1.f, 1.f, 1.f}, sn1[4] = {0.f, 0.f, 0.f, 0.f};
    load_heads<T, N>(x, ahead, u, H, more, r1);
    load_heads<T, N>(dy, ahead, u, H, more, g1);
    if (more) load_turn(a, p1, u, cs1, sn1);
    const Walk now = w;
    w = ahead;
    ahead.next(a, m);
    if (ahead.item < items) p1 = ahead.position(a);
#pragma unroll
    for (int i = 0; i < 4; ++i) sn[i] = -sn[i];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool here = now.item < items && u.on && now.c * N + i < H;
      float v[8], d[8], sq = 0.f, gn = 0.f;
      r[i].get(v);
      g[i].get(d);
      if (u.rot) rotate(d, cs, sn, PAIRS);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sq = fmaf(v[j], v[j], sq);
        gn = fmaf(d[j] * wt[j], v[j], gn);
      }
      const float rs = rsqrtf(group_sum<G>(sq) / (float)a.D + a.eps);
      const float mean = group_sum<G>(gn) * rs / (float)a.D;  // mean(g n)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v[j] * rs;
        dw[j] += here ? d[j] * n : 0.f;
        v[j] = rs * (d[j] * wt[j] - n * mean);
      }
      if (here) store8<T>(dx.row(now.b, now.t, now.c * N + i), u.lo, u.hi, v);
      r[i] = r1[i];
      g[i] = g1[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = cs1[i], sn[i] = sn1[i];
    lead += w.step;
  }
  // groups of the block, in order
  __shared__ float red[kThreads * 8];
#pragma unroll
  for (int j = 0; j < 8; ++j) red[j * kThreads + threadIdx.x] = dw[j];
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * G; i += kThreads) {
    const int lane = i % G, j = i / G;
    const Unit v = unit_of(lane, a);
    if (!v.on) continue;
    float s = 0.f;
    for (int k = 0; k < NG; ++k) s += red[j * kThreads + k * G + lane];
    a.part[(int64_t)blockIdx.x * a.D + (j < 4 ? v.lo + j : v.hi + j - 4)] = s;
  }
}

// Columns of the partial sums, one block per (queries or keys, 32 columns): 32
// lanes of columns by 32 slices of blocks, the slices then added in order.
__global__ void __launch_bounds__(1024) qknorm_dw_kernel(const QkArgs a) {
  const int m = blockIdx.y, lane = threadIdx.x % 32, col = blockIdx.x * 32 + lane, sl = threadIdx.x / 32;
  if (!a.dw[m]) return;
  __shared__ float red[32][33];
  const float* p = a.part + (int64_t)(m ? a.blocks[0] : 0) * a.D + col;
  float s = 0.f;
  if (col < a.D) {
#pragma unroll 4
    for (int k = sl; k < a.blocks[m]; k += 32) s += p[(int64_t)k * a.D];
  }
  red[sl][lane] = s;
  __syncthreads();
  if (sl == 0 && col < a.D) {
    for (int k = 1; k < 32; ++k) s += red[k][lane];
    a.dw[m][col] = s;
  }
}

// Blocks of a walk: as many as stay resident (four or five an SM), shared between
// queries and keys by their numbers of items; a block more where one side has few.
constexpr int kFwdBlocks = 152 * 5, kBwdBlocks = 152 * 4;

void share_blocks(QkArgs* a, int groups, int most) {
  const int64_t items[2] = {a->BT * a->chunks[0], a->BT * a->chunks[1]};
  for (int m = 0; m < 2; ++m) {
    const int64_t need = (items[m] + groups - 1) / groups;
    const int64_t part = most * items[m] / (items[0] + items[1]);
    a->blocks[m] = (int)(need < part ? need : part > 0 ? part : need > 0 ? 1 : 0);
  }
}

int group_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

template <typename T, int G>
cudaError_t qk_launch_g(QkArgs a, bool fwd, cudaStream_t s) {
  const int heads = fwd ? kFwdHeads : kBwdHeads;
  for (int m = 0; m < 2; ++m) a.chunks[m] = (a.H[m] + heads - 1) / heads;
  share_blocks(&a, kThreads / G, fwd ? kFwdBlocks : kBwdBlocks);
  const int blocks = a.blocks[0] + a.blocks[1];
  if (fwd) {
    if (a.pairs) qknorm_fwd_kernel<T, G, true><<<blocks, kThreads, 0, s>>>(a);
    else qknorm_fwd_kernel<T, G, false><<<blocks, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  if (a.pairs) qknorm_bwd_kernel<T, G, true><<<blocks, kThreads, 0, s>>>(a);
  else qknorm_bwd_kernel<T, G, false><<<blocks, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
  qknorm_dw_kernel<<<dim3((a.D + 31) / 32, 2), 1024, 0, s>>>(a);
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
  if (B > (1LL << 31) || T > (1LL << 31) || B * T > (1LL << 40)) return SCAN_ERR_UNSUPPORTED;
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
  return (size_t)(kBwdBlocks + 2) * (size_t)D * 4;
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
