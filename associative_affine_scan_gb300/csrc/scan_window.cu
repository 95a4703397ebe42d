// scan_window.cu -- attention with a sliding window and a few first tokens that
// stay visible: the entry points and the general kernels.
//
//   s_ij = scale q_i k_j where key j is seen: j <= i and (i - j < W or j < S)
//   p_ij = exp(s_ij - lse_i), lse_i = log sum_j exp(s_ij), o_i = sum_j p_ij v_j
//   delta_i = do_i o_i, ds_ij = p_ij (do_i v_j - delta_i) scale
//   dq_i = sum_j ds_ij k_j, dk_j = sum_i ds_ij q_i, dv_j = sum_i p_ij do_i
//
// Query heads h G .. h G + G - 1 share key head h; dk and dv are sums over them.
// Queries are the last Tq of Tk positions; a query before the first key sees
// nothing: o = 0, lse = -inf, and its gradients are 0.
//
// The kernels here serve fp32 operands and operands that tensor copies cannot
// address. They are tiles of 32 rows by 32 rows in shared memory and fp32
// multiply-adds, four threads a row: bound by the shared-memory reads of the
// products. Only tiles with a seen pair are visited. 8 x 128 queries of 16 heads of 128
// and a window of 256 take 470 us in bf16, where the tensor-core kernel takes 18 us.
#include "scan_mixer.h"
#include "scan_window_step.h"
#include "scan_window_tc.h"

namespace scan {
namespace {

constexpr int kTile = 32;

template <typename T>
__device__ __forceinline__ View<T> vw(const scan_view4& v) {
  return View<T>{static_cast<T*>(v.ptr), v.stride_b, v.stride_t, v.stride_h};
}

// Rows [t0, t0 + 32) of one head into shared memory as fp32, zeros from `end` on.
template <typename T, int D1>
__device__ __forceinline__ void load_tile(float* dst, const View<const T>& v, int64_t b, int64_t t0,
                                          int64_t end, int64_t h, int D) {
  for (int i = threadIdx.x; i < kTile * D; i += blockDim.x) {
    const int r = i / D, c = i % D;
    dst[r * D1 + c] = t0 + r < end ? to_f32(v.row(b, t0 + r, h)[c]) : 0.f;
  }
}

__device__ __forceinline__ bool seen(int64_t i, int64_t j, const WinArgs& a) {
  return j <= i && (i - j < a.W || j < a.S);
}

constexpr int kLd = kMixMaxDim + 1;  // row pitch: rows of a column lie in different banks
constexpr int kColsT = kMixMaxDim / 4;

template <typename T>
__global__ void __launch_bounds__(4 * kTile) window_fwd_general(const WinArgs a) {
  extern __shared__ float sm[];
  float *sq = sm, *sk = sq + kTile * kLd, *sv = sk + kTile * kLd, *sp = sv + kTile * kLd;
  if (a.cu && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    check_seqlens(a.cu, a.n_seqs, a.Tq, a.hdr);
  TileRows g;
  if (!tile_rows(a.cu, a.n_seqs, a.Tq, a.Tk, blockIdx.x, kTile, &g)) return;
  const int h = blockIdx.y % a.Hq, hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.y / a.Hq;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
  const View<const T> q = vw<const T>(a.q), k = vw<const T>(a.k), v = vw<const T>(a.v);
  load_tile<T, kLd>(sq, q, b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D);
  const int64_t i = g.off + g.t0 + r;
  const KeyTiles kt = key_tiles(g.off + g.t0, g.off + g.t0 + kTile - 1, g.nk, a.W, a.S, kTile);
  float m = -INFINITY, l = 0.f, o[kColsT];
#pragma unroll
  for (int x = 0; x < kColsT; ++x) o[x] = 0.f;
  for (int64_t n = 0; n < kt.count(); ++n) {
    const int64_t j0 = kt.at(n) * kTile;
    __syncthreads();
    load_tile<T, kLd>(sk, k, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    load_tile<T, kLd>(sv, v, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    __syncthreads();
    float s[8], mx = -INFINITY;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = c + 4 * x;
      float e = 0.f;
      for (int d = 0; d < a.D; ++d) e = fmaf(sq[r * kLd + d], sk[j * kLd + d], e);
      s[x] = seen(i, j0 + j, a) && j0 + j < g.nk ? e * a.scale : -INFINITY;
      mx = fmaxf(mx, s[x]);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const float mn = fmaxf(m, mx);
    const float base = mn == -INFINITY ? 0.f : mn;  // no key seen so far: every weight is 0
    const float keep = expf(m - base);
    float sum = 0.f;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float e = expf(s[x] - base);
      sp[r * (kTile + 1) + c + 4 * x] = e;
      sum += e;
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    l = l * keep + sum;
    m = mn;
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kColsT; ++x) {
      if (4 * x < a.D) {
        float e = o[x] * keep;
        for (int j = 0; j < kTile; ++j) e = fmaf(sp[r * (kTile + 1) + j], sv[j * kLd + c + 4 * x], e);
        o[x] = e;
      }
    }
  }
  if (g.t0 + r >= g.nq) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;  // l is 0 where no key is seen; NaN stays
  T* out = vw<T>(a.o).row(b, g.qbeg + g.t0 + r, h);
#pragma unroll
  for (int x = 0; x < kColsT; ++x)
    if (4 * x < a.D) out[c + 4 * x] = from_f32<T>(o[x] * inv);
  if (c == 0) a.lse[(b * a.Hq + h) * a.Tq + g.qbeg + g.t0 + r] = l == 0.f ? -INFINITY : m + logf(l);
}

// delta_i = sum_d dout o of every query row: one warp a row.
template <typename T>
__global__ void __launch_bounds__(256) window_delta_kernel(const WinArgs a, int64_t rows) {
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

template <typename T>
__global__ void __launch_bounds__(4 * kTile) window_dq_general(const WinArgs a) {
  extern __shared__ float sm[];
  float *sq = sm, *sd = sq + kTile * kLd, *sk = sd + kTile * kLd, *sv = sk + kTile * kLd,
        *sp = sv + kTile * kLd;
  TileRows g;
  if (!tile_rows(a.cu, a.n_seqs, a.Tq, a.Tk, blockIdx.x, kTile, &g)) return;
  const int h = blockIdx.y % a.Hq, hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.y / a.Hq;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
  const View<const T> q = vw<const T>(a.q), k = vw<const T>(a.k), v = vw<const T>(a.v),
                      dout = vw<const T>(a.dout);
  load_tile<T, kLd>(sq, q, b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D);
  load_tile<T, kLd>(sd, dout, b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D);
  const int64_t i = g.off + g.t0 + r;
  const bool live = g.t0 + r < g.nq;
  const int64_t st = (b * a.Hq + h) * a.Tq + g.qbeg + g.t0 + r;
  const float lse = live ? a.lse[st] : -INFINITY, delta = live ? a.delta[st] : 0.f;
  const KeyTiles kt = key_tiles(g.off + g.t0, g.off + g.t0 + kTile - 1, g.nk, a.W, a.S, kTile);
  float o[kColsT];
#pragma unroll
  for (int x = 0; x < kColsT; ++x) o[x] = 0.f;
  for (int64_t n = 0; n < kt.count(); ++n) {
    const int64_t j0 = kt.at(n) * kTile;
    __syncthreads();
    load_tile<T, kLd>(sk, k, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    load_tile<T, kLd>(sv, v, b, g.kbeg + j0, g.kbeg + g.nk, hk, a.D);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int j = c + 4 * x;
      float e = 0.f, f = 0.f;
      for (int d = 0; d < a.D; ++d) {
        e = fmaf(sq[r * kLd + d], sk[j * kLd + d], e);
        f = fmaf(sd[r * kLd + d], sv[j * kLd + d], f);
      }
      float ds = 0.f;
      if (live && seen(i, j0 + j, a) && j0 + j < g.nk)
        ds = expf(e * a.scale - lse) * (f - delta) * a.scale;
      sp[r * (kTile + 1) + j] = ds;
    }
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kColsT; ++x)
      if (4 * x < a.D)
        for (int j = 0; j < kTile; ++j)
          o[x] = fmaf(sp[r * (kTile + 1) + j], sk[j * kLd + c + 4 * x], o[x]);
  }
  if (!live) return;
  T* out = vw<T>(a.dq).row(b, g.qbeg + g.t0 + r, h);
#pragma unroll
  for (int x = 0; x < kColsT; ++x)
    if (4 * x < a.D) out[c + 4 * x] = from_f32<T>(o[x]);
}

// A tile of keys against every query that sees it, over the heads that share it.
template <typename T>
__global__ void __launch_bounds__(4 * kTile) window_dkv_general(const WinArgs a) {
  extern __shared__ float sm[];
  float *sk = sm, *sv = sk + kTile * kLd, *sq = sv + kTile * kLd, *sd = sq + kTile * kLd,
        *sp = sd + kTile * kLd, *ss = sp + kTile * (kTile + 1), *st = ss + kTile * (kTile + 1);
  if (a.cu && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    check_seqlens(a.cu, a.n_seqs, a.Tk, a.hdr);
  TileRows g;
  if (!tile_rows(a.cu, a.n_seqs, a.Tq, a.Tk, blockIdx.x, kTile, &g)) return;
  const int hk = blockIdx.y % a.Hk, G = a.Hq / a.Hk;
  const int64_t b = blockIdx.y / a.Hk;
  const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
  const View<const T> q = vw<const T>(a.q), k = vw<const T>(a.k), v = vw<const T>(a.v),
                      dout = vw<const T>(a.dout);
  load_tile<T, kLd>(sk, k, b, g.kbeg + g.t0, g.kbeg + g.nk, hk, a.D);
  load_tile<T, kLd>(sv, v, b, g.kbeg + g.t0, g.kbeg + g.nk, hk, a.D);
  const int64_t j = g.t0 + r;
  // queries (as rows of the sequence) that may see a key of this tile
  const int64_t kend = g.t0 + kTile < g.nk ? g.t0 + kTile : g.nk;
  int64_t lo = g.t0 - g.off, hi = kend - 1 + a.W - 1 - g.off;
  if (g.t0 < a.S || hi > g.nq - 1) hi = g.nq - 1;
  lo = lo < 0 ? 0 : lo;
  float dk[kColsT], dv[kColsT];
#pragma unroll
  for (int x = 0; x < kColsT; ++x) dk[x] = dv[x] = 0.f;
  for (int hh = 0; hh < G; ++hh) {
    const int h = hk * G + hh;
    for (int64_t t = lo / kTile * kTile; t <= hi; t += kTile) {
      __syncthreads();
      load_tile<T, kLd>(sq, q, b, g.qbeg + t, g.qbeg + g.nq, h, a.D);
      load_tile<T, kLd>(sd, dout, b, g.qbeg + t, g.qbeg + g.nq, h, a.D);
      if (threadIdx.x < kTile) {
        const int64_t at = (b * a.Hq + h) * a.Tq + g.qbeg + t + threadIdx.x;
        const bool live = t + threadIdx.x < g.nq;
        st[threadIdx.x] = live ? a.lse[at] : -INFINITY;
        st[kTile + threadIdx.x] = live ? a.delta[at] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const int i = c + 4 * x;
        float e = 0.f, f = 0.f;
        for (int d = 0; d < a.D; ++d) {
          e = fmaf(sk[r * kLd + d], sq[i * kLd + d], e);
          f = fmaf(sv[r * kLd + d], sd[i * kLd + d], f);
        }
        float p = 0.f;
        if (t + i < g.nq && j < g.nk && seen(g.off + t + i, j, a)) p = expf(e * a.scale - st[i]);
        sp[r * (kTile + 1) + i] = p;
        ss[r * (kTile + 1) + i] = p * (f - st[kTile + i]) * a.scale;
      }
      __syncwarp();
#pragma unroll
      for (int x = 0; x < kColsT; ++x)
        if (4 * x < a.D)
          for (int i = 0; i < kTile; ++i) {
            dv[x] = fmaf(sp[r * (kTile + 1) + i], sd[i * kLd + c + 4 * x], dv[x]);
            dk[x] = fmaf(ss[r * (kTile + 1) + i], sq[i * kLd + c + 4 * x], dk[x]);
          }
    }
  }
  if (j >= g.nk) return;
  T* ok = vw<T>(a.dk).row(b, g.kbeg + j, hk);
  T* ov = vw<T>(a.dv).row(b, g.kbeg + j, hk);
#pragma unroll
  for (int x = 0; x < kColsT; ++x)
    if (4 * x < a.D) {
      ok[c + 4 * x] = from_f32<T>(dk[x]);
      ov[c + 4 * x] = from_f32<T>(dv[x]);
    }
}

template <typename T>
cudaError_t general_fwd(const WinArgs& a, cudaStream_t s) {
  const size_t smem = (3 * kTile * kLd + kTile * (kTile + 1)) * 4;
  cudaError_t e = cudaFuncSetAttribute(window_fwd_general<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (a.Tq + kTile - 1) / kTile + (a.cu ? a.n_seqs : 0);
  window_fwd_general<T><<<dim3((unsigned)tiles, (unsigned)(a.B * a.Hq)), 4 * kTile, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t delta_launch(const WinArgs& a, cudaStream_t s) {
  const int64_t rows = a.B * a.Tq * a.Hq;
  if (rows > 0) window_delta_kernel<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a, rows);
  return cudaGetLastError();
}

template <typename T>
cudaError_t general_bwd(const WinArgs& a, cudaStream_t s) {
  const size_t sq = (4 * kTile * kLd + kTile * (kTile + 1)) * 4;
  const size_t skv = (4 * kTile * kLd + 2 * kTile * (kTile + 1) + 2 * kTile) * 4;
  cudaError_t e = cudaFuncSetAttribute(window_dq_general<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sq);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(window_dkv_general<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)skv);
  if (e == cudaSuccess) e = delta_launch<T>(a, s);
  if (e != cudaSuccess) return e;
  const int64_t extra = a.cu ? a.n_seqs : 0;
  const int64_t tq = (a.Tq + kTile - 1) / kTile + extra, tk = (a.Tk + kTile - 1) / kTile + extra;
  if (tq > 0) window_dq_general<T><<<dim3((unsigned)tq, (unsigned)(a.B * a.Hq)), 4 * kTile, sq, s>>>(a);
  if (tk > 0) window_dkv_general<T><<<dim3((unsigned)tk, (unsigned)(a.B * a.Hk)), 4 * kTile, skv, s>>>(a);
  return cudaGetLastError();
}

bool given(const scan_view4* v) { return v && v->ptr; }

scan_status win_common(WinArgs* a, scan_dtype dt, int64_t Hq, int64_t Hk, int64_t D, int32_t n_seqs) {
  if (dt != SCAN_F32 && dt != SCAN_BF16) return SCAN_ERR_INVALID_ARG;
  if (a->B < 0 || a->Tq < 0 || a->Tk < 0 || Hq < 0 || Hk < 0 || D < 1 || n_seqs < 0)
    return SCAN_ERR_INVALID_ARG;
  if (a->W < 1 || a->S < 0 || !(a->scale > 0.f) || !(a->scale < INFINITY)) return SCAN_ERR_INVALID_ARG;
  if (Hk == 0 ? Hq != 0 : Hq % Hk != 0) return SCAN_ERR_INVALID_ARG;
  if (a->cu && (a->B != 1 || a->Tq != a->Tk || (n_seqs == 0 && a->Tq > 0))) return SCAN_ERR_INVALID_ARG;
  if (D > kMixMaxDim || D % 8) return SCAN_ERR_UNSUPPORTED;
  if (Hq > 65535 || a->B > 65535 || a->B * Hq > 65535 || a->Tq > 0x7fffffffLL || a->Tk > 0x7fffffffLL)
    return SCAN_ERR_UNSUPPORTED;
  // positions are at most 2^31: larger windows see everything
  if (a->W > (1LL << 32)) a->W = 1LL << 32;
  if (a->S > (1LL << 32)) a->S = 1LL << 32;
  a->Hq = (int)Hq;
  a->Hk = (int)Hk;
  a->D = (int)D;
  a->n_seqs = n_seqs;
  return SCAN_OK;
}

scan_status win_workspace(WinArgs* a, void* ws, size_t bytes, size_t need) {
  if (!ws || (uintptr_t)ws % 16 || bytes < need) return SCAN_ERR_WORKSPACE;
  a->hdr = static_cast<WsHeader*>(ws);
  a->ws = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeaderBytes);
  return SCAN_OK;
}

// ---------------------------------------------------------------------------
// one token a request over a ring of S + W cached keys, any operands

// One block a (request, query head), eight warps that take every eighth key.
template <typename T>
__global__ void __launch_bounds__(256) window_step_general(const WinStepArgs a) {
  const int h = (int)(blockIdx.x % a.Hq), G = a.Hq / a.Hk, hk = h / G;
  const int64_t b = blockIdx.x / a.Hq;
  const int64_t slot = a.slots ? (int64_t)a.slots[b] : b, pos = a.pos[b];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  T* o = static_cast<T*>(a.o.ptr) + b * a.o.stride_b + h * a.o.stride_h;
  if (slot < 0 || slot >= a.n_slots || pos < 0) {
    for (int d = threadIdx.x; d < a.D; d += 256) o[d] = from_f32<T>(0.f);
    return;
  }
  const int64_t at = pos < a.S ? pos : a.S + (pos - a.S) % a.W;
  const int64_t n = pos + 1 < a.cap ? pos + 1 : a.cap;
  const int64_t row = (int64_t)a.Hk * a.D;
  T* kc = static_cast<T*>(a.kc) + slot * a.cap * row + (int64_t)hk * a.D;
  T* vc = static_cast<T*>(a.vc) + slot * a.cap * row + (int64_t)hk * a.D;
  const T* q = static_cast<const T*>(a.q.ptr) + b * a.q.stride_b + h * a.q.stride_h;
  const T* kn = static_cast<const T*>(a.k.ptr) + b * a.k.stride_b + hk * a.k.stride_h;
  const T* vn = static_cast<const T*>(a.v.ptr) + b * a.v.stride_b + hk * a.v.stride_h;
  if (h % G == 0)  // the new token's row is read from k and v, never from the cache
    for (int d = threadIdx.x; d < a.D; d += 256) {
      kc[at * row + d] = kn[d];
      vc[at * row + d] = vn[d];
    }
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < 4; ++x) qv[x] = lane + 32 * x < a.D ? to_f32(q[lane + 32 * x]) : 0.f;
  for (int64_t j = warp; j < n; j += 8) {
    const T* kr = j == at ? kn : kc + j * row;
    const T* vr = j == at ? vn : vc + j * row;
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

}  // namespace

cudaError_t launch_window_general_fwd(const WinArgs& a, scan_dtype dt, cudaStream_t s) {
  return dt == SCAN_BF16 ? general_fwd<__nv_bfloat16>(a, s) : general_fwd<float>(a, s);
}
cudaError_t launch_window_general_bwd(const WinArgs& a, scan_dtype dt, cudaStream_t s) {
  return dt == SCAN_BF16 ? general_bwd<__nv_bfloat16>(a, s) : general_bwd<float>(a, s);
}

}  // namespace scan

using namespace scan;

extern "C" {

size_t window_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                                   int64_t D, int64_t window, int64_t sinks, int64_t n_seqs,
                                   int32_t backward) {
  if (B < 0 || Tq < 0 || Tk < 0 || Hq < 0 || Hk < 0 || D < 1 || D > kMixMaxDim || window < 1 ||
      sinks < 0 || n_seqs < 0)
    return 0;
  if (!backward) return kWsHeaderBytes;
  return kWsHeaderBytes + round_up((size_t)(B * Hq * Tq) * 4, 256) +
         window_tc_bwd_floats(B, Tq, Tk, Hk, D, window, sinks, n_seqs > 0) * 4;
}

scan_status window_attn_fwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                            const int32_t* cu_seqlens, int32_t n_seqs, const scan_view4* o,
                            float* lse, int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk,
                            int64_t D, int64_t window, int64_t sinks, float scale, scan_dtype dt,
                            void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  WinArgs a{};
  a.cu = cu_seqlens;
  a.B = B;
  a.Tq = Tq;
  a.Tk = Tk;
  a.W = window;
  a.S = sinks;
  a.scale = scale;
  scan_status st = win_common(&a, dt, Hq, Hk, D, cu_seqlens ? n_seqs : 0);
  if (st != SCAN_OK) return st;
  if (B * Tq * Hq == 0) return SCAN_OK;
  if (!given(q) || !given(o) || !lse || (Tk > 0 && (!given(k) || !given(v))))
    return SCAN_ERR_INVALID_ARG;
  st = win_workspace(&a, workspace, workspace_bytes,
                     window_attn_workspace_bytes(B, Tq, Tk, Hq, Hk, D, window, sinks, a.n_seqs, 0));
  if (st != SCAN_OK) return st;
  a.q = *q;
  if (Tk > 0) a.k = *k, a.v = *v;
  a.o = *o;
  a.lse = lse;
  const cudaError_t e = window_tc_fits(a, dt, false) ? launch_window_tc_fwd(a, stream)
                                                     : launch_window_general_fwd(a, dt, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status window_attn_bwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                            const scan_view4* o, const float* lse, const scan_view4* dout,
                            const int32_t* cu_seqlens, int32_t n_seqs, const scan_view4* dq,
                            const scan_view4* dk, const scan_view4* dv, int64_t B, int64_t Tq,
                            int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t window,
                            int64_t sinks, float scale, scan_dtype dt, void* workspace,
                            size_t workspace_bytes, cudaStream_t stream) {
  WinArgs a{};
  a.cu = cu_seqlens;
  a.B = B;
  a.Tq = Tq;
  a.Tk = Tk;
  a.W = window;
  a.S = sinks;
  a.scale = scale;
  scan_status st = win_common(&a, dt, Hq, Hk, D, cu_seqlens ? n_seqs : 0);
  if (st != SCAN_OK) return st;
  if (B * Hq * (Tq + Tk) == 0) return SCAN_OK;
  if (Tq > 0 && (!given(q) || !given(o) || !given(dout) || !given(dq) || !lse))
    return SCAN_ERR_INVALID_ARG;
  if (Tk > 0 && (!given(k) || !given(v) || !given(dk) || !given(dv))) return SCAN_ERR_INVALID_ARG;
  st = win_workspace(&a, workspace, workspace_bytes,
                     window_attn_workspace_bytes(B, Tq, Tk, Hq, Hk, D, window, sinks, a.n_seqs, 1));
  if (st != SCAN_OK) return st;
  if (Tq > 0) a.q = *q, a.o = *o, a.dout = *dout, a.dq = *dq;
  if (Tk > 0) a.k = *k, a.v = *v, a.dk = *dk, a.dv = *dv;
  a.lse = const_cast<float*>(lse);
  a.delta = a.ws;
  cudaError_t e;
  if (window_tc_fits(a, dt, true))
    e = launch_window_tc_bwd(a, a.ws + round_up((size_t)(B * Hq * Tq) * 4, 256) / 4, stream);
  else
    e = launch_window_general_bwd(a, dt, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status window_attn_step(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                             void* k_cache, void* v_cache, const int32_t* positions,
                             const int32_t* slots, int64_t n_slots, const scan_view4* o, int64_t B,
                             int64_t Hq, int64_t Hk, int64_t D, int64_t window, int64_t sinks,
                             float scale, scan_dtype dt, cudaStream_t stream) {
  WinArgs c{};
  c.B = B;
  c.W = window;
  c.S = sinks;
  c.scale = scale;
  const scan_status st = win_common(&c, dt, Hq, Hk, D, 0);
  if (st != SCAN_OK) return st;
  if (n_slots < 0) return SCAN_ERR_INVALID_ARG;
  if (B * Hq == 0) return SCAN_OK;
  if (!given(q) || !given(k) || !given(v) || !given(o) || !k_cache || !v_cache || !positions)
    return SCAN_ERR_INVALID_ARG;
  if (!slots && n_slots < B) return SCAN_ERR_INVALID_ARG;
  if ((uintptr_t)k_cache % 16 || (uintptr_t)v_cache % 16) return SCAN_ERR_ALIGNMENT;
  if (window + sinks > 0x7fffffffLL) return SCAN_ERR_UNSUPPORTED;
  WinStepArgs a{*q, *k, *v, *o, k_cache, v_cache, slots, positions, n_slots, window + sinks,
                window, sinks, (int)Hq, (int)Hk, (int)D, scale};
  if (window_step_fits(a, dt)) return launch_window_step(a, B, stream) == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
  if (dt == SCAN_BF16) window_step_general<__nv_bfloat16><<<(unsigned)(B * Hq), 256, 0, stream>>>(a);
  else window_step_general<float><<<(unsigned)(B * Hq), 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // extern "C"
