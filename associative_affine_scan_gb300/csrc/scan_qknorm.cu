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
// One read and one write of every element forward, two reads and one write
// backward, about ten operations on each. A row of D elements is held by the 8, 16
// or 32 lanes that cover it, eight elements a lane, so the norm's sum is three to
// five shuffles and no row is read twice. A lane's eight elements are four pairs
// (elements 4u.. and R/2 + 4u.., or 8u.. where neighbours are paired), so the rotation
// needs no exchange, and go through the arithmetic two at a time. A group of lanes
// takes four heads of one token (two in fp32): the token's cosines and sines are read
// once for them. A block has either queries or keys; the backward's walk over the
// tokens, with their weight's gradient in registers. What hides the latency of DRAM is
// the number of rows in flight: they stay in their own type until they are used.
//
// Forward of 8 x 4096 tokens, 16 + 4 heads of 128, bf16: 57 us, 5.9 TB/s, bound by
// DRAM. Backward: 95 us, 5.3 TB/s, bound half by DRAM and half by the issue of
// instructions (scalar arithmetic and two heads a group: 116 us). A ring of
// asynchronous copies to shared memory, two items ahead, took 175 us, and the next
// item's rows in registers 145 us: a lane's copies of 8 bytes and what they spill cost
// more than the latency that they hide.
#include "scan_mixer.h"
#include "scan_tc.cuh"

namespace scan {
namespace {

using tc::add2;
using tc::fma2;
using tc::mul2;

constexpr int kThreads = 256;
// Heads of one token that a group of lanes takes: 64 bytes of each operand a lane.
// What an item costs besides (its place, pointers, table entries) is shared by them:
// the backward of 8 x 4096 x 20 heads of 128 in bf16 took 137 / 117 / 100 / 112 us with
// 1 / 2 / 4 / 8, each at its best block size and number of blocks.
template <typename T>
constexpr int kHeads = sizeof(T) == 2 ? 4 : 2;

// Division of numbers below 2^31 by a fixed divisor: one high product, one add and
// one shift (Granlund and Montgomery, "Division by invariant integers using
// multiplication").
struct Divisor {
  uint32_t d, mul;
  int shift;
  void set(int64_t by) {
    d = (uint32_t)by;
    shift = 0;
    while ((1LL << shift) < by) ++shift;
    mul = (uint32_t)((((1ULL << shift) - (uint64_t)by) << 32) / (uint64_t)by + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(mul, n) + n) >> shift; }
};

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
  int blocks[2];  // blocks of the queries, and of the keys
  int narrow;     // items fit 31 bits
  Divisor by_chunks[2], by_T;
  float inv_D;
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
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
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
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    const uint32_t u[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* row, int lo, int hi, const float2 (&v)[4]);
template <>
__device__ __forceinline__ void store8<float>(float* row, int lo, int hi, const float2 (&v)[4]) {
  *reinterpret_cast<float4*>(row + lo) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  *reinterpret_cast<float4*>(row + hi) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* row, int lo, int hi,
                                                      const float2 (&v)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
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
__device__ __forceinline__ void rotate(float2 (&v)[4], const float (&c)[4], const float (&s)[4],
                                       bool pairs) {
  if (pairs) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = fma2(v[i], make_float2(c[i], c[i]), mul2(make_float2(v[i].y, v[i].x), make_float2(-s[i], s[i])));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = v[i], y = v[2 + i], ci = make_float2(c[2 * i], c[2 * i + 1]);
      v[i] = fma2(x, ci, mul2(y, make_float2(-s[2 * i], -s[2 * i + 1])));
      v[2 + i] = fma2(y, ci, mul2(x, make_float2(s[2 * i], s[2 * i + 1])));
    }
  }
}

// Sums of both numbers over a group of lanes.
template <int G>
__device__ __forceinline__ float2 group_sum(float2 v) {
#pragma unroll
  for (int d = G / 2; d; d >>= 1)
    v = add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d)));
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
  c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
  s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
  if (!ok) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = s[i] = __int_as_float(0x7fc00000);
  }
}

__device__ __forceinline__ void load_weight(const float* w, const Unit& u, float2 (&v)[4]) {
  Raw<float> r;
  if (w && u.on) {
    r.load(w, u.lo, u.hi);
    r.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(1.f, 1.f);
  }
}

// What an item (one token, N heads of the queries or the keys) is.
struct Item {
  int64_t tok, b, t;
  int h;
};
template <int N>
__device__ __forceinline__ Item item_at(const QkArgs& a, int m, int64_t i) {
  Item r;
  const int per = a.chunks[m];
  if (a.narrow) {
    const uint32_t tok = (m ? a.by_chunks[1] : a.by_chunks[0])((uint32_t)i), b = a.by_T(tok);
    r.tok = tok;
    r.h = (int)((uint32_t)i - tok * per) * N;
    r.b = b;
    r.t = tok - b * (uint32_t)a.T;
  } else {
    r.tok = i / per;
    r.h = (int)(i - r.tok * per) * N;
    r.b = r.tok / a.T;
    r.t = r.tok - r.b * a.T;
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void load_heads(const View<const T>& x, const Item& w, const Unit& u, int H, bool live,
                                           Raw<T> (&r)[N]) {
  const T* p = x.row(w.b, w.t, w.h);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    r[i].clear();
    if (live && u.on && w.h + i < H) r[i].load(p + i * x.sh, u.lo, u.hi);
  }
}

template <typename T>
__device__ __forceinline__ View<T> qk_view(const scan_view4& v) {
  return View<T>{static_cast<T*>(v.ptr), v.stride_b, v.stride_t, v.stride_h};
}

template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 4) qknorm_fwd_kernel(const QkArgs a) {
  constexpr int N = kHeads<T>;
  const int m = blockIdx.x >= a.blocks[0];
  const int64_t block = m ? blockIdx.x - a.blocks[0] : blockIdx.x;
  const int64_t i0 = block * (kThreads / G) + threadIdx.x / G;
  const bool live = i0 < a.BT * a.chunks[m];  // lanes of a dead group stay for the shuffles
  const Item w = item_at<N>(a, m, live ? i0 : 0);
  const Unit u = unit_of(threadIdx.x % G, a);
  const int H = a.H[m];
  const int64_t p = a.pos ? (int64_t)a.pos[w.tok] : w.t;
  Raw<T> r[N];
  load_heads<T, N>(m ? qk_view<const T>(a.x[1]) : qk_view<const T>(a.x[0]), w, u, H, live, r);
  float2 wt[4];
  float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
  load_weight(a.w[m], u, wt);
  load_turn(a, p, u, cs, sn);
  const View<T> y = m ? qk_view<T>(a.y[1]) : qk_view<T>(a.y[0]);
  T* out = y.row(w.b, w.t, w.h);
  float2 rs[N / 2];  // of two heads each
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 v[4], sq = make_float2(0.f, 0.f);
    r[i].get(v);
#pragma unroll
    for (int j = 0; j < 4; ++j) sq = fma2(v[j], v[j], sq);
    (i % 2 ? rs[i / 2].y : rs[i / 2].x) = sq.x + sq.y;
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) rs[i] = group_sum<G>(rs[i]);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float f = rsqrtf(fmaf(i % 2 ? rs[i / 2].y : rs[i / 2].x, a.inv_D, a.eps));
    const float2 f2 = make_float2(f, f);
    float2 v[4];
    r[i].get(v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], mul2(wt[j], f2));
    if (u.rot) rotate(v, cs, sn, PAIRS);
    if (live && u.on && w.h + i < H) store8<T>(out + i * y.sh, u.lo, u.hi, v);
  }
}

// Each block walks tokens with its weight's gradient in registers and leaves one
// partial sum; the partial sums are added in block order by the kernel below, so
// the result does not depend on the order in which blocks finish.
template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) qknorm_bwd_kernel(const QkArgs a) {
  constexpr int N = kHeads<T>, NG = kThreads / G;
  const int m = blockIdx.x >= a.blocks[0];
  const int64_t block = m ? blockIdx.x - a.blocks[0] : blockIdx.x;
  const int64_t items = a.BT * a.chunks[m], step = (int64_t)a.blocks[m] * NG;
  const Unit u = unit_of(threadIdx.x % G, a);
  const View<const T> x = m ? qk_view<const T>(a.x[1]) : qk_view<const T>(a.x[0]);
  const View<const T> dy = m ? qk_view<const T>(a.dy[1]) : qk_view<const T>(a.dy[0]);
  const View<T> dx = m ? qk_view<T>(a.dx[1]) : qk_view<T>(a.dx[0]);
  const int H = a.H[m];
  float2 wt[4], dw[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) dw[j] = make_float2(0.f, 0.f);
  load_weight(a.w[m], u, wt);
  // whole warps leave together: the bound is on the warp's first group
  int64_t lead = block * NG + (threadIdx.x / 32) * (32 / G), i0 = lead + (threadIdx.x % 32) / G;
  Item w = item_at<N>(a, m, i0 < items ? i0 : 0);
  int64_t p = a.pos ? (int64_t)a.pos[w.tok] : w.t;
  for (; lead < items; lead += step) {
    const bool live = i0 < items;
    Raw<T> r[N], g[N];
    load_heads<T, N>(x, w, u, H, live, r);
    load_heads<T, N>(dy, w, u, H, live, g);
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    load_turn(a, p, u, cs, sn);
#pragma unroll
    for (int i = 0; i < 4; ++i) sn[i] = -sn[i];
    T* out = dx.row(w.b, w.t, w.h);
    const int h = w.h;
    i0 += step;  // the next position now: its table entries depend on it
    w = item_at<N>(a, m, i0 < items ? i0 : 0);
    p = a.pos ? (int64_t)a.pos[w.tok] : w.t;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool some = live && h + i < H, here = some && u.on;
      float2 v[4], d[4], e[4], sq = make_float2(0.f, 0.f), gn = sq;
      r[i].get(v);
      g[i].get(d);
      if (u.rot) rotate(d, cs, sn, PAIRS);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        e[j] = mul2(d[j], wt[j]);
        sq = fma2(v[j], v[j], sq);
        gn = fma2(e[j], v[j], gn);
      }
      const float2 sum = group_sum<G>(make_float2(sq.x + sq.y, gn.x + gn.y));
      // a row that is not there is zeros and adds nothing, also where eps is 0
      const float rs = some ? rsqrtf(fmaf(sum.x, a.inv_D, a.eps)) : 0.f;
      const float back = -(sum.y * a.inv_D) * rs * rs * rs;  // -r^2 mean(g n) of each x
      const float2 rs2 = make_float2(rs, rs), back2 = make_float2(back, back);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dw[j] = fma2(mul2(d[j], rs2), v[j], dw[j]);
        v[j] = fma2(v[j], back2, mul2(e[j], rs2));
      }
      if (here) store8<T>(out + i * dx.sh, u.lo, u.hi, v);
    }
  }
  // groups of the block, in order
  __shared__ float red[kThreads * 8];
#pragma unroll
  for (int j = 0; j < 8; ++j) red[j * kThreads + threadIdx.x] = j % 2 ? dw[j / 2].y : dw[j / 2].x;
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
// lanes of columns by 32 slices of blocks, the slices then added in order. 6 us, the
// latency of ten dependent rounds of loads and sums.
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

// Blocks of the backward's walk: what stays resident, shared between queries and
// keys by their numbers of items.
constexpr int kBwdBlocks = 152 * 2;

void share_blocks(QkArgs* a, int groups, bool fwd) {
  const int64_t items[2] = {a->BT * a->chunks[0], a->BT * a->chunks[1]};
  for (int m = 0; m < 2; ++m) {
    const int64_t need = (items[m] + groups - 1) / groups;
    const int64_t part = kBwdBlocks * items[m] / (items[0] + items[1]);
    a->blocks[m] = (int)(fwd || need < part ? need : part > 0 ? part : need > 0 ? 1 : 0);
  }
  a->narrow = items[0] < (1LL << 31) && items[1] < (1LL << 31) && a->T < (1LL << 31);
  if (a->narrow) {
    for (int m = 0; m < 2; ++m) a->by_chunks[m].set(a->chunks[m] > 0 ? a->chunks[m] : 1);
    a->by_T.set(a->T);
  }
}

int group_lanes(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

template <typename T, int G>
cudaError_t qk_launch_g(QkArgs a, bool fwd, cudaStream_t s) {
  constexpr int heads = kHeads<T>;
  for (int m = 0; m < 2; ++m) a.chunks[m] = (a.H[m] + heads - 1) / heads;
  share_blocks(&a, kThreads / G, fwd);
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
  if (B * T * ((Hq + 1) / 2 + (Hk + 1) / 2) / 8 >= 0x7fffffffLL) return SCAN_ERR_UNSUPPORTED;  // grid.x
  if (R > 0 && B * T > 0 && (!cs || !sn || P < 1)) return SCAN_ERR_INVALID_ARG;
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
  a->inv_D = 1.f / (float)D;
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
