// scan_cross.cu -- attention to the states of another sequence, of another length
// (an encoder's): the entry points and the general kernels.
//
//   s_ij = scale q_i k_j over the n keys of the row's sequence
//   p_ij = exp(s_ij - lse_i), lse_i = log sum_j exp(s_ij), o_i = sum_j p_ij v_j
//   delta_i = do_i o_i, ds_ij = p_ij (do_i v_j - delta_i) scale
//   dq_i = sum_j ds_ij k_j, dk_j = sum_i ds_ij q_i, dv_j = sum_i p_ij do_i
//
// Query heads h G .. h G + G - 1 share key head h; dk and dv are sums over them. A
// sequence of no keys gives o = 0, lse = -inf and zero gradients.
//
// The kernels here serve fp32 operands and operands that tensor copies cannot
// address: tiles of 64 by 64 in shared memory, four by four products a thread in fp32
// multiply-adds. An operand that is summed over its columns lies transposed, so that
// both factors are read 16 bytes at a time: three shared-memory cycles a warp for 16
// multiply-adds a thread.
#include "scan_cross.h"
#include "scan_cross_tc.h"

namespace scan {
namespace {

constexpr int kTile = 64;
constexpr int kPitch = kTile + 4;
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ View<T> vw(const scan_view4& v) {
  return View<T>{static_cast<T*>(v.ptr), v.stride_b, v.stride_t, v.stride_h};
}

// Rows [t0, t0 + 64) of one head as fp32, zeros from row `end` and column D on:
// transposed (d, row), or as they lie (row, d).
template <typename T, int DP>
__device__ __forceinline__ void load_t(float* dst, const View<const T>& v, int64_t b, int64_t t0, int64_t end, int64_t h,
                                       int D) {
  const int r = threadIdx.x % kTile;
  const bool on = t0 + r < end;
  const T* const p = v.row(b, on ? t0 + r : t0, h);
#pragma unroll 8
  for (int c = threadIdx.x / kTile; c < DP; c += kThreads / kTile)
    dst[c * kPitch + r] = on && c < D ? to_f32(p[c]) : 0.f;
}
template <typename T, int DP>
__device__ __forceinline__ void load_r(float* dst, const View<const T>& v, int64_t b, int64_t t0, int64_t end, int64_t h,
                                       int D) {
#pragma unroll 8
  for (int i = threadIdx.x; i < kTile * DP; i += kThreads) {
    const int r = i / DP, c = i % DP;
    dst[i] = t0 + r < end && c < D ? to_f32(v.row(b, t0 + r, h)[c]) : 0.f;
  }
}

__device__ __forceinline__ float4 ld4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// acc[i][j] += sum over d of a[d][4 ty + i] b[d][4 tx + j].
template <int DP>
__device__ __forceinline__ void product_tt(float (&acc)[4][4], const float* a, const float* b, int ty, int tx) {
#pragma unroll 8
  for (int d = 0; d < DP; ++d) {
    const float4 x = ld4(a + d * kPitch + 4 * ty), y = ld4(b + d * kPitch + 4 * tx);
    const float u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
  }
}
// acc[i][h][j] += sum over k of p[k][4 ty + i] m[k][64 h + 4 tx + j], 64 rows k.
template <int DP>
__device__ __forceinline__ void product_pm(float (&acc)[4][DP / 64][4], const float* p, const float* m, int ty, int tx) {
#pragma unroll 4
  for (int k = 0; k < kTile; ++k) {
    const float4 x = ld4(p + k * kPitch + 4 * ty);
    const float u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int h = 0; h < DP / 64; ++h) {
      const float4 y = ld4(m + k * DP + 64 * h + 4 * tx);
      const float v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][h][j] = fmaf(u[i], v[j], acc[i][h][j]);
    }
  }
}
// A thread's 4 x 4 of a tile, transposed into shared memory.
__device__ __forceinline__ void store_t(float* dst, const float (&s)[4][4], int ty, int tx) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<float4*>(dst + (4 * tx + j) * kPitch + 4 * ty) = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
}
template <typename T, int DP>
__device__ __forceinline__ void write_rows(const View<T>& out, const float (&acc)[4][DP / 64][4], int64_t b, int64_t t0,
                                           int64_t end, int64_t h, int D, const float (&f)[4], int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + 4 * ty + i;
    if (t >= end) continue;
    T* const row = out.row(b, t, h);
#pragma unroll
    for (int x = 0; x < DP / 64; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (64 * x + 4 * tx + j < D) row[64 * x + 4 * tx + j] = from_f32<T>(acc[i][x][j] * f[i]);
  }
}
// The 16 threads of a row are half a warp.
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) cross_fwd_general(const CrossArgs a) {
  extern __shared__ float4 raw[];
  float *const sq = reinterpret_cast<float*>(raw), *const sk = sq + DP * kPitch, *const sv = sk + DP * kPitch;
  float* const sp = sk;  // the weights, once the scores are formed
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  CrossRows g;
  const int h = blockIdx.y % a.Hq, hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.y / a.Hq;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kTile, false, &g)) return;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const View<const T> q = vw<const T>(a.q), k = vw<const T>(a.k), v = vw<const T>(a.v);
  load_t<T, DP>(sq, q, b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D);
  float m[4], l[4], o[4][DP / 64][4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int64_t j0 = 0; j0 < g.nk; j0 += kTile) {
    __syncthreads();
    load_t<T, DP>(sk, k, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    load_r<T, DP>(sv, v, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    __syncthreads();
    float s[4][4] = {};
    product_tt<DP>(s, sq, sk, ty, tx);
    __syncthreads();
    float keep[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = j0 + 4 * tx + j < g.nk ? s[i][j] * a.scale : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      const float mn = fmaxf(m[i], row_max(top)), base = mn == -INFINITY ? 0.f : mn;
      keep[i] = expf(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) sum += s[i][j] = expf(s[i][j] - base);
      l[i] = l[i] * keep[i] + row_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int x = 0; x < DP / 64; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][x][j] *= keep[i];
    }
    store_t(sp, s, ty, tx);
    __syncthreads();
    product_pm<DP>(o, sp, sv, ty, tx);
  }
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = l[i] == 0.f ? 0.f : 1.f / l[i];  // l is 0 where there is no key; NaN stays
    const int64_t t = g.t0 + 4 * ty + i;
    if (tx == 0 && t < g.nq)
      a.lse[(b * a.Hq + h) * a.Tq + g.qbeg + t] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
  }
  write_rows<T, DP>(vw<T>(a.o), o, b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D, f, ty, tx);
}

// delta_i = sum_d dout o of every query row: one warp a row.
template <typename T>
__global__ void __launch_bounds__(256) cross_delta_general(const CrossArgs a, int64_t rows) {
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (w >= rows) return;
  const int h = (int)(w % a.Hq);
  const int64_t t = (w / a.Hq) % a.Tq, b = w / a.Hq / a.Tq;
  const T* o = vw<const T>(a.o).row(b, t, h);
  const T* d = vw<const T>(a.dout).row(b, t, h);
  float s = 0.f;
  for (int c = threadIdx.x % 32; c < a.D; c += 32) s = fmaf(to_f32(o[c]), to_f32(d[c]), s);
#pragma unroll
  for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
  if (threadIdx.x % 32 == 0) a.delta[(b * a.Hq + h) * a.Tq + t] = s;
}

// A tile of queries against every key.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) cross_dq_general(const CrossArgs a) {
  extern __shared__ float4 raw[];
  float *const sq = reinterpret_cast<float*>(raw), *const sd = sq + DP * kPitch, *const sb = sd + DP * kPitch,
                *const sp = sb + DP * kPitch;
  CrossRows g;
  const int h = blockIdx.y % a.Hq, hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.y / a.Hq;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kTile, false, &g)) return;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const View<const T> k = vw<const T>(a.k), v = vw<const T>(a.v);
  load_t<T, DP>(sq, vw<const T>(a.q), b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D);
  load_t<T, DP>(sd, vw<const T>(a.dout), b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D);
  float lse[4], delta[4], dq[4][DP / 64][4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = g.t0 + 4 * ty + i, at = (b * a.Hq + h) * a.Tq + g.qbeg + t;
    lse[i] = t < g.nq ? a.lse[at] : INFINITY;
    delta[i] = t < g.nq ? a.delta[at] : 0.f;
  }
  for (int64_t j0 = 0; j0 < g.nk; j0 += kTile) {
    __syncthreads();
    load_t<T, DP>(sb, v, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    __syncthreads();
    float dp[4][4] = {}, s[4][4] = {};
    product_tt<DP>(dp, sd, sb, ty, tx);
    __syncthreads();
    load_t<T, DP>(sb, k, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    __syncthreads();
    product_tt<DP>(s, sq, sb, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = j0 + 4 * tx + j < g.nk ? expf(s[i][j] * a.scale - lse[i]) * (dp[i][j] - delta[i]) : 0.f;
    __syncthreads();
    store_t(sp, s, ty, tx);
    load_r<T, DP>(sb, k, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    __syncthreads();
    product_pm<DP>(dq, sp, sb, ty, tx);
  }
  const float f[4] = {a.scale, a.scale, a.scale, a.scale};
  write_rows<T, DP>(vw<T>(a.dq), dq, b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D, f, ty, tx);
}

// A tile of keys against every query, over the heads that share it. Rows past a
// sequence's keys (padding) get zeros.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) cross_dkv_general(const CrossArgs a) {
  extern __shared__ float4 raw[];
  float *const sk = reinterpret_cast<float*>(raw), *const sv = sk + DP * kPitch, *const sb = sv + DP * kPitch,
                *const sp = sb + DP * kPitch, *const ss = sp + kTile * kPitch;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  CrossRows g;
  const int hk = blockIdx.y % a.Hk, G = a.Hq / a.Hk;
  const int64_t b = blockIdx.y / a.Hk;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kTile, true, &g)) return;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  const View<const T> q = vw<const T>(a.q), dout = vw<const T>(a.dout);
  load_t<T, DP>(sk, vw<const T>(a.k), b, g.kbeg + g.t0, g.kbeg + g.nk, hk, a.D);
  load_t<T, DP>(sv, vw<const T>(a.v), b, g.kbeg + g.t0, g.kbeg + g.nk, hk, a.D);
  float dk[4][DP / 64][4] = {}, dv[4][DP / 64][4] = {};
  const int64_t nq = g.t0 < g.nk ? g.nq : 0;
  for (int hh = 0; hh < G; ++hh) {
    const int h = hk * G + hh;
    for (int64_t t0 = 0; t0 < nq; t0 += kTile) {
      __syncthreads();
      load_t<T, DP>(sb, dout, b, g.qbeg + t0, g.qbeg + nq, h, a.D);
      __syncthreads();
      float dp[4][4] = {}, s[4][4] = {};
      product_tt<DP>(dp, sv, sb, ty, tx);
      __syncthreads();
      load_t<T, DP>(sb, q, b, g.qbeg + t0, g.qbeg + nq, h, a.D);
      __syncthreads();
      product_tt<DP>(s, sk, sb, ty, tx);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t t = t0 + 4 * tx + j, at = (b * a.Hq + h) * a.Tq + g.qbeg + t;
        const float lse = t < nq ? a.lse[at] : INFINITY, delta = t < nq ? a.delta[at] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[i][j] = t < nq && g.t0 + 4 * ty + i < g.nk ? expf(s[i][j] * a.scale - lse) : 0.f;
          dp[i][j] = s[i][j] * (dp[i][j] - delta);
        }
      }
      store_t(sp, s, ty, tx);
      store_t(ss, dp, ty, tx);
      __syncthreads();
      load_r<T, DP>(sb, dout, b, g.qbeg + t0, g.qbeg + nq, h, a.D);
      __syncthreads();
      product_pm<DP>(dv, sp, sb, ty, tx);
      __syncthreads();
      load_r<T, DP>(sb, q, b, g.qbeg + t0, g.qbeg + nq, h, a.D);
      __syncthreads();
      product_pm<DP>(dk, ss, sb, ty, tx);
    }
  }
  const int64_t rows = a.cu_q ? g.nk : a.Tk;
  const float one[4] = {1.f, 1.f, 1.f, 1.f}, f[4] = {a.scale, a.scale, a.scale, a.scale};
  write_rows<T, DP>(vw<T>(a.dk), dk, b, g.kbeg + g.t0, g.kbeg + rows, hk, a.D, f, ty, tx);
  write_rows<T, DP>(vw<T>(a.dv), dv, b, g.kbeg + g.t0, g.kbeg + rows, hk, a.D, one, ty, tx);
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int DP>
cudaError_t general_fwd(const CrossArgs& a, cudaStream_t s) {
  const size_t smem = (2 * DP * kPitch + kTile * DP) * 4;
  static_assert(DP >= kTile, "the weights fit the keys' place");
  const cudaError_t e = allow_smem(cross_fwd_general<T, DP>, smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.Tq + kTile - 1) / kTile + (a.cu_q ? a.n_seqs : 0);
  cross_fwd_general<T, DP><<<dim3((unsigned)tiles, (unsigned)(a.B * a.Hq)), kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t general_bwd(const CrossArgs& a, cudaStream_t s) {
  const size_t sq = (3 * DP * kPitch + kTile * kPitch) * 4, skv = sq + kTile * kPitch * 4;
  cudaError_t e = allow_smem(cross_dq_general<T, DP>, sq);
  if (e == cudaSuccess) e = allow_smem(cross_dkv_general<T, DP>, skv);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.B * a.Tq * a.Hq, extra = a.cu_q ? a.n_seqs : 0;
  const int64_t tq = (a.Tq + kTile - 1) / kTile + extra, tk = (a.Tk + kTile - 1) / kTile + extra;
  if (rows > 0) {
    cross_delta_general<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a, rows);
    cross_dq_general<T, DP><<<dim3((unsigned)tq, (unsigned)(a.B * a.Hq)), kThreads, sq, s>>>(a);
  }
  if (a.Tk > 0) cross_dkv_general<T, DP><<<dim3((unsigned)tk, (unsigned)(a.B * a.Hk)), kThreads, skv, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// one query token a request, any operands: one block a (request, query head), eight
// warps that take every eighth key

template <typename T>
__global__ void __launch_bounds__(256) cross_step_general(const CrossStepArgs a) {
  const int h = (int)(blockIdx.x % a.Hq), hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.x / a.Hq;
  const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  T* const o = static_cast<T*>(a.o.ptr) + b * a.o.stride_b + h * a.o.stride_h;
  const int64_t n = slot < 0 || slot >= a.n_slots ? 0 : keys_of(a.lens, slot, a.Tk);
  if (n == 0) {  // an idle request, or no keys
    for (int d = threadIdx.x; d < a.D; d += 256) o[d] = from_f32<T>(0.f);
    return;
  }
  const T* const k = vw<const T>(a.k).row(slot, 0, hk);
  const T* const v = vw<const T>(a.v).row(slot, 0, hk);
  const T* const q = static_cast<const T*>(a.q.ptr) + b * a.q.stride_b + h * a.q.stride_h;
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) qv[x] = lane + 32 * x < a.D ? to_f32(q[lane + 32 * x]) : 0.f;
  for (int64_t j = warp; j < n; j += 8) {
    const T* const kr = k + j * a.k.stride_t;
    const T* const vr = v + j * a.v.stride_t;
    float s = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (lane + 32 * x < a.D) s = fmaf(qv[x], to_f32(kr[lane + 32 * x]), s);
#pragma unroll
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale;
    const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
    const float keep = expf(m - base), p = expf(s - base);
    l = l * keep + p;
    m = mn;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (lane + 32 * x < a.D) acc[x] = fmaf(p, to_f32(vr[lane + 32 * x]), acc[x] * keep);
  }
  __shared__ float sm[8], sl[8], sa[8][kMixMaxDim];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int x = 0; x < 4; ++x) sa[warp][lane + 32 * x] = acc[x];
  __syncthreads();
  if (threadIdx.x < a.D) {
    float mx = -INFINITY;
    for (int w = 0; w < 8; ++w) mx = fmaxf(mx, sm[w]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, e = 0.f;
    for (int w = 0; w < 8; ++w) {
      const float f = expf(sm[w] - base);
      sum = fmaf(sl[w], f, sum);
      e = fmaf(sa[w][threadIdx.x], f, e);
    }
    o[threadIdx.x] = from_f32<T>(e / sum);
  }
}

bool given(const scan_view4* v) { return v && v->ptr; }

scan_status cross_sizes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, float scale,
                        scan_dtype dt) {
  if (dt != SCAN_F32 && dt != SCAN_BF16) return SCAN_ERR_INVALID_ARG;
  if (B < 0 || Tq < 0 || Tk < 0 || Hq < 0 || Hk < 0 || D < 1) return SCAN_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return SCAN_ERR_INVALID_ARG;
  if (Hk == 0 ? Hq != 0 : Hq % Hk != 0) return SCAN_ERR_INVALID_ARG;
  if (D > kMixMaxDim || D % 8) return SCAN_ERR_UNSUPPORTED;
  if (Hq > 65535 || B > 65535 || B * Hq > 65535 || Tq > 0x7fffffffLL || Tk > 0x7fffffffLL)
    return SCAN_ERR_UNSUPPORTED;
  if (B * Hq * Tq > (1LL << 33)) return SCAN_ERR_UNSUPPORTED;  // blocks of the row sums
  return SCAN_OK;
}

scan_status cross_common(CrossArgs* a, const int32_t* lens, const int32_t* cu_q, const int32_t* cu_k, int32_t n_seqs,
                         int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, float scale,
                         scan_dtype dt) {
  const scan_status st = cross_sizes(B, Tq, Tk, Hq, Hk, D, scale, dt);
  if (st != SCAN_OK) return st;
  if (n_seqs < 0 || !cu_q != !cu_k || (cu_q && lens)) return SCAN_ERR_INVALID_ARG;
  if (cu_q && (B != 1 || (n_seqs == 0 && Tq + Tk > 0))) return SCAN_ERR_INVALID_ARG;
  *a = CrossArgs{};
  a->lens = lens;
  a->cu_q = cu_q;
  a->cu_k = cu_k;
  a->n_seqs = cu_q ? n_seqs : 0;
  a->B = B;
  a->Tq = Tq;
  a->Tk = Tk;
  a->Hq = (int)Hq;
  a->Hk = (int)Hk;
  a->D = (int)D;
  a->scale = scale;
  return SCAN_OK;
}

scan_status cross_workspace(CrossArgs* a, void* ws, size_t bytes, size_t need) {
  if (!ws || (uintptr_t)ws % 16 || bytes < need) return SCAN_ERR_WORKSPACE;
  a->hdr = static_cast<WsHeader*>(ws);
  a->delta = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeaderBytes);
  a->ws = a->delta + round_up((size_t)(a->B * a->Hq * a->Tq) * 4, 256) / 4;
  return SCAN_OK;
}

}  // namespace

cudaError_t launch_cross_general_fwd(const CrossArgs& a, scan_dtype dt, cudaStream_t s) {
  if (dt == SCAN_BF16) return a.D <= 64 ? general_fwd<__nv_bfloat16, 64>(a, s) : general_fwd<__nv_bfloat16, 128>(a, s);
  return a.D <= 64 ? general_fwd<float, 64>(a, s) : general_fwd<float, 128>(a, s);
}
cudaError_t launch_cross_general_bwd(const CrossArgs& a, scan_dtype dt, cudaStream_t s) {
  if (dt == SCAN_BF16) return a.D <= 64 ? general_bwd<__nv_bfloat16, 64>(a, s) : general_bwd<__nv_bfloat16, 128>(a, s);
  return a.D <= 64 ? general_bwd<float, 64>(a, s) : general_bwd<float, 128>(a, s);
}

}  // namespace scan

using namespace scan;

extern "C" {

size_t cross_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t n_seqs,
                                  int32_t backward) {
  if (B < 0 || Tq < 0 || Tk < 0 || Hq < 0 || Hk < 0 || D < 1 || D > kMixMaxDim || n_seqs < 0) return 0;
  if (!backward) return kWsHeaderBytes;
  return kWsHeaderBytes + round_up((size_t)(B * Hq * Tq) * 4, 256) + cross_tc_bwd_floats(B, Tq, Tk, Hq, D, n_seqs) * 4;
}

scan_status cross_attn_fwd(const scan_view4* q, const scan_view4* k, const scan_view4* v, const int32_t* k_lens,
                           const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t n_seqs,
                           const scan_view4* o, float* lse, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                           int64_t D, float scale, scan_dtype dt, void* workspace, size_t workspace_bytes,
                           cudaStream_t stream) {
  CrossArgs a;
  scan_status st = cross_common(&a, k_lens, cu_seqlens_q, cu_seqlens_k, n_seqs, B, Tq, Tk, Hq, Hk, D, scale, dt);
  if (st != SCAN_OK) return st;
  if (B * Tq * Hq == 0) return SCAN_OK;
  if (!given(q) || !given(o) || !lse || (Tk > 0 && (!given(k) || !given(v)))) return SCAN_ERR_INVALID_ARG;
  st = cross_workspace(&a, workspace, workspace_bytes, cross_attn_workspace_bytes(B, Tq, Tk, Hq, Hk, D, a.n_seqs, 0));
  if (st != SCAN_OK) return st;
  a.q = *q;
  if (Tk > 0) a.k = *k, a.v = *v;
  a.o = *o;
  a.lse = lse;
  const cudaError_t e = cross_tc_fits(a, dt, false) ? launch_cross_tc_fwd(a, stream)
                                                    : launch_cross_general_fwd(a, dt, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status cross_attn_bwd(const scan_view4* q, const scan_view4* k, const scan_view4* v, const scan_view4* o,
                           const float* lse, const scan_view4* dout, const int32_t* k_lens,
                           const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t n_seqs,
                           const scan_view4* dq, const scan_view4* dk, const scan_view4* dv, int64_t B, int64_t Tq,
                           int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, float scale, scan_dtype dt, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
  CrossArgs a;
  scan_status st = cross_common(&a, k_lens, cu_seqlens_q, cu_seqlens_k, n_seqs, B, Tq, Tk, Hq, Hk, D, scale, dt);
  if (st != SCAN_OK) return st;
  if (B * Hq * (Tq + Tk) == 0) return SCAN_OK;
  if (Tq > 0 && (!given(q) || !given(o) || !given(dout) || !given(dq) || !lse)) return SCAN_ERR_INVALID_ARG;
  if (Tk > 0 && (!given(k) || !given(v) || !given(dk) || !given(dv))) return SCAN_ERR_INVALID_ARG;
  st = cross_workspace(&a, workspace, workspace_bytes, cross_attn_workspace_bytes(B, Tq, Tk, Hq, Hk, D, a.n_seqs, 1));
  if (st != SCAN_OK) return st;
  if (Tq > 0) a.q = *q, a.o = *o, a.dout = *dout, a.dq = *dq;
  if (Tk > 0) a.k = *k, a.v = *v, a.dk = *dk, a.dv = *dv;
  a.lse = const_cast<float*>(lse);
  const cudaError_t e = cross_tc_fits(a, dt, true) ? launch_cross_tc_bwd(a, stream)
                                                   : launch_cross_general_bwd(a, dt, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

size_t cross_attn_step_workspace_bytes(int64_t B, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D) {
  if (B < 0 || Tk < 0 || Hq < 0 || Hk < 0 || D < 1 || D > kMixMaxDim) return 0;
  return kWsHeaderBytes + cross_step_bytes(B, Tk, Hq, Hk, D);
}

scan_status cross_attn_step(const scan_view4* q, const scan_view4* k_cache, const scan_view4* v_cache,
                            const int32_t* lens, const int32_t* slots, int64_t n_slots, const scan_view4* o, int64_t B,
                            int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, float scale, scan_dtype dt, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  const scan_status st = cross_sizes(B, 1, Tk, Hq, Hk, D, scale, dt);
  if (st != SCAN_OK) return st;
  if (n_slots < 0 || (!slots && n_slots < B)) return SCAN_ERR_INVALID_ARG;
  if (B * Hq == 0) return SCAN_OK;
  if (!given(q) || !given(o) || (n_slots * Tk > 0 && (!given(k_cache) || !given(v_cache)))) return SCAN_ERR_INVALID_ARG;
  if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < cross_attn_step_workspace_bytes(B, Tk, Hq, Hk, D))
    return SCAN_ERR_WORKSPACE;
  CrossStepArgs a{*q, {}, {}, *o, lens, slots, n_slots, Tk, (int)Hq, (int)Hk, (int)D, scale,
                  static_cast<WsHeader*>(workspace), static_cast<char*>(workspace) + kWsHeaderBytes};
  if (n_slots * Tk > 0) a.k = *k_cache, a.v = *v_cache;
  if (cross_step_fits(a, dt, B)) return launch_cross_step(a, B, stream) == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
  if (dt == SCAN_BF16) cross_step_general<__nv_bfloat16><<<(unsigned)(B * Hq), 256, 0, stream>>>(a);
  else cross_step_general<float><<<(unsigned)(B * Hq), 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // extern "C"
