// scan_residual.cu -- the norms before and after a block of a network, fused with
// the block's gate, dropout and residual scale, forward and backward.
//
//   z  = w_post y r,  r = (mean(y^2) + eps)^(-1/2)      (z = y without w_post)
//   x' = alpha x + drop(gate z)                          the stream after the block
//   n  = w_next x' q, q = (mean(x'^2) + eps)^(-1/2)      what the next block reads
// n is the norm of x' as it is stored, so that the backward, which reads x', is the
// gradient of what the forward computed. With dx', dn the gradients of x' and n:
//   e  = w_next dn,  G = dx' + q (e - x' q^2 mean(e x')),  dx = alpha G
//   u  = drop(G),    f = w_post gate u,  dy = r (f - y r^2 mean(f y))
//   dw_next = sum dn x' q;  h = sum u y r over rows that share a gate:
//   dgate = w_post h,  dw_post = sum over gates of gate h
// so two sums a column, not three, leave the walk over the rows.
//
// Two reads and two writes of each element forward, four and two backward, some ten
// and thirty operations: bound by DRAM. A row is held by the 32 to 512 threads that
// cover it, eight elements a thread (or two times eight), so that no row is read
// twice; sums are shuffles and one exchange through shared memory.
#include "scan_mixer.h"
#include "scan_philox.cuh"

namespace scan {
namespace {

struct NormArgs {
  const void *x, *y, *dxo, *dn;  // forward: x, y; backward: x', y, dx', dn
  void *xo, *n, *dx, *dy;
  int64_t x_sb, x_st, y_sb, y_st, xo_sb, xo_st, n_sb, n_st;  // (backward: xo = dx', n = dn)
  int64_t dx_sb, dx_st, dy_sb, dy_st;
  const float *w_post, *gate, *w_next;  // nullable
  int64_t gate_sb;                      // C where each batch row has a gate, else 0
  int64_t B, T, rows;
  int C, W;          // W: warps a row
  float alpha, eps, inv_C;
  Drop drop;
  // backward
  float *part_h, *part_n;  // [units][C]
  int64_t groups, span;    // rows that share a gate: `groups` runs of `span` rows
  int chunks;              // units a group
  int row_gate;
};

// Eight elements of a row, in memory and as numbers.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *(reinterpret_cast<float4*>(p) + 1) = b;
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
};

// Weights of eight columns, ones where there are none.
__device__ __forceinline__ void weights(const float* w, int c, bool on, float (&v)[8]) {
  Eight<float> e;
  if (w && on) {
    e.load(w + c);
    e.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.f;
  }
}

// Sums of N numbers over the W warps of a row, in warp order, for all its threads.
// `red`: one slot a warp of the block; every thread of the block comes here.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*red)[4], int W) {
#pragma unroll
  for (int d = 16; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
  if (W == 1) return;
  const int warp = threadIdx.x / 32, first = warp / W * W;
  if (threadIdx.x % 32 == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp][i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = 0.f;
  for (int w = 0; w < W; ++w)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += red[first + w][i];
}

// u = drop(u) of the eight elements of block `block` of the tensor.
__device__ __forceinline__ void dropped(float (&v)[8], const Drop& d, uint64_t block, uint64_t call, uint64_t seed) {
  const uint4 r = philox(block, call, seed);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = kept_low(w[i], d.limit) ? v[2 * i] * d.scale : 0.f;
    v[2 * i + 1] = kept_high(w[i], d.limit) ? v[2 * i + 1] * d.scale : 0.f;
  }
}

// V: vectors of eight elements a thread.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(512) residual_fwd_kernel(const NormArgs a) {
  __shared__ float red[2][32][4];
  const int per = blockDim.x / 32 / a.W, lane = threadIdx.x % (32 * a.W);  // rows a block, place in the row
  const int64_t row = (int64_t)blockIdx.x * per + threadIdx.x / (32 * a.W);
  const bool live = row < a.rows;
  const int64_t b = live ? row / a.T : 0, t = live ? row - b * a.T : 0;
  const X* const x = static_cast<const X*>(a.x) + b * a.x_sb + t * a.x_st;
  const Y* const y = static_cast<const Y*>(a.y) + b * a.y_sb + t * a.y_st;
  Eight<X> ex[V];
  Eight<Y> ey[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (lane + v * 32 * a.W);
    ex[v].clear();
    ey[v].clear();
    if (live && c < a.C) {
      ex[v].load(x + c);
      if (a.y) ey[v].load(y + c);
    }
  }
  if (a.y) {
    uint64_t seed, call;
    a.drop.read(&seed, &call);
    float r = 1.f;
    if (a.w_post) {
      float s[1] = {0.f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        ey[v].get(f);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = fmaf(f[i], f[i], s[0]);
      }
      row_sums(s, red[0], a.W);
      r = rsqrtf(fmaf(s[0], a.inv_C, a.eps));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (lane + v * 32 * a.W);
      const bool on = live && c < a.C;
      float f[8], g[8], w[8];
      ey[v].get(f);
      weights(a.w_post, c, on, w);
      weights(a.gate ? a.gate + b * a.gate_sb : nullptr, c, on, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * w[i] * g[i];
      if (a.drop.limit) dropped(f, a.drop, (uint64_t)(row * (a.C / 8) + c / 8), call, seed);
      ex[v].get(g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = fmaf(a.alpha, g[i], f[i]);
      ex[v].set(f);
      if (on) ex[v].store(static_cast<X*>(a.xo) + b * a.xo_sb + t * a.xo_st + c);
    }
  }
  if (!a.w_next) return;
  float s[1] = {0.f};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float f[8];
    ex[v].get(f);
    if (8 * (lane + v * 32 * a.W) < a.C)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] = fmaf(f[i], f[i], s[0]);
  }
  row_sums(s, red[1], a.W);
  const float q = rsqrtf(fmaf(s[0], a.inv_C, a.eps));
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (lane + v * 32 * a.W);
    const bool on = live && c < a.C;
    float f[8], w[8];
    ex[v].get(f);
    weights(a.w_next, c, on, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * q * w[i];
    Eight<Y> e;
    e.set(f);
    if (on) e.store(static_cast<Y*>(a.n) + b * a.n_sb + t * a.n_st + c);
  }
}

// A block walks units: a part of the rows that share a gate, its column sums in
// registers, left in the workspace and added in order by the kernel below.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(512) residual_bwd_kernel(const NormArgs a) {
  __shared__ float red[2][32][4];
  extern __shared__ float fold[];  // [rows a block - 1][2][C]
  const int per = blockDim.x / 32 / a.W, lane = threadIdx.x % (32 * a.W), mine = threadIdx.x / (32 * a.W);
  const int64_t units = a.groups * a.chunks;
  uint64_t seed, call;
  a.drop.read(&seed, &call);
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t grp = unit / a.chunks, ch = unit - grp * a.chunks;
    const int64_t beg = grp * a.span + a.span * ch / a.chunks, end = grp * a.span + a.span * (ch + 1) / a.chunks;
    const float* const gate = a.gate ? a.gate + (a.row_gate ? grp * a.gate_sb : 0) : nullptr;
    float h[V][8], dw[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[v][i] = dw[v][i] = 0.f;
    for (int64_t r0 = beg; r0 < end; r0 += per) {
      const int64_t row = r0 + mine;
      const bool live = row < end;
      const int64_t b = live ? row / a.T : 0, t = live ? row - b * a.T : 0;
      Eight<X> ex[V], eg[V];
      Eight<Y> ey[V], en[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (lane + v * 32 * a.W);
        ex[v].clear();
        eg[v].clear();
        ey[v].clear();
        en[v].clear();
        if (live && c < a.C) {
          if (a.w_next) {
            ex[v].load(static_cast<const X*>(a.x) + b * a.x_sb + t * a.x_st + c);
            en[v].load(static_cast<const Y*>(a.dn) + b * a.n_sb + t * a.n_st + c);
          }
          if (a.dxo) eg[v].load(static_cast<const X*>(a.dxo) + b * a.xo_sb + t * a.xo_st + c);
          if (a.y) ey[v].load(static_cast<const Y*>(a.y) + b * a.y_sb + t * a.y_st + c);
        }
      }
      float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (lane + v * 32 * a.W);
        float y[8], x[8], e[8], w[8];
        ey[v].get(y);
        ex[v].get(x);
        en[v].get(e);
        weights(a.w_next, c, c < a.C, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = fmaf(y[i], y[i], s[0]);
          s[1] = fmaf(x[i], x[i], s[1]);
          s[2] = fmaf(e[i] * w[i], x[i], s[2]);
        }
      }
      row_sums(s, red[0], a.W);
      // a row that is not there is zeros and adds nothing, also where eps is 0
      const float r = !a.w_post ? 1.f : live ? rsqrtf(fmaf(s[0], a.inv_C, a.eps)) : 0.f;
      const float q = live && a.w_next ? rsqrtf(fmaf(s[1], a.inv_C, a.eps)) : 0.f;
      const float mean = s[2] * a.inv_C * q;  // of e x' q
      float f[V][8], s2[1] = {0.f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (lane + v * 32 * a.W);
        const bool on = live && c < a.C;
        float x[8], e[8], w[8], g[8];
        ex[v].get(x);
        en[v].get(e);
        eg[v].get(g);
        weights(a.w_next, c, on, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= q;
          dw[v][i] = fmaf(e[i], x[i], dw[v][i]);
          g[i] = fmaf(q, fmaf(x[i], -mean, e[i] * w[i]), g[i]);
        }
        Eight<X> out;
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = a.alpha * g[i];
        out.set(e);
        if (on) out.store(static_cast<X*>(a.dx) + b * a.dx_sb + t * a.dx_st + c);
        if (a.y) {
          if (a.drop.limit) dropped(g, a.drop, (uint64_t)(row * (a.C / 8) + c / 8), call, seed);
          float y[8];
          ey[v].get(y);
          weights(a.w_post, c, on, w);
          weights(gate, c, on, e);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[v][i] = fmaf(g[i], y[i] * r, h[v][i]);
            f[v][i] = g[i] * w[i] * e[i];
            s2[0] = fmaf(f[v][i], y[i], s2[0]);
          }
        }
      }
      if (a.y) {
        if (a.w_post) row_sums(s2, red[1], a.W);
        const float mean2 = a.w_post ? s2[0] * a.inv_C * r : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = 8 * (lane + v * 32 * a.W);
          float y[8];
          ey[v].get(y);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[v][i] = r * fmaf(y[i] * r, -mean2, f[v][i]);
          Eight<Y> out;
          out.set(f[v]);
          if (live && c < a.C) out.store(static_cast<Y*>(a.dy) + b * a.dy_sb + t * a.dy_st + c);
        }
      }
      if (!a.y || !a.w_post) __syncthreads();  // `red` is free again
    }
    // the block's rows, in order
    if (per > 1) {
      __syncthreads();
      if (mine > 0)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = 8 * (lane + v * 32 * a.W);
          if (c < a.C)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              fold[((mine - 1) * 2) * a.C + c + i] = h[v][i];
              fold[((mine - 1) * 2 + 1) * a.C + c + i] = dw[v][i];
            }
        }
      __syncthreads();
    }
    if (mine == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = 8 * (lane + v * 32 * a.W);
        if (c >= a.C) continue;
        for (int k = 0; k < per - 1; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            h[v][i] += fold[(k * 2) * a.C + c + i];
            dw[v][i] += fold[(k * 2 + 1) * a.C + c + i];
          }
        Eight<float> e;
        e.set(h[v]);
        e.store(a.part_h + unit * a.C + c);
        e.set(dw[v]);
        e.store(a.part_n + unit * a.C + c);
      }
    if (per > 1) __syncthreads();
  }
}

struct SumArgs {
  const float *part_h, *part_n, *w_post, *gate;
  float *dw_post, *dgate, *dw_next;
  int64_t units;
  int C, chunks, row_gate;
};

// Columns of the partial sums: 32 lanes of columns by 32 slices of units, the slices
// then added in order. blockIdx.y 0: dw_next; 1: dw_post and a shared gate's gradient.
__global__ void __launch_bounds__(1024) residual_sums_kernel(const SumArgs a) {
  const int lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane, sl = threadIdx.x / 32;
  if (blockIdx.y == 0 ? !a.dw_next : !a.dw_post && (!a.dgate || a.row_gate)) return;
  __shared__ float red[32][33];
  const float* p = (blockIdx.y ? a.part_h : a.part_n) + c;
  const bool scaled = blockIdx.y && a.row_gate;
  float s = 0.f;
  if (c < a.C) {
#pragma unroll 4
    for (int64_t k = sl; k < a.units; k += 32)
      s += scaled ? a.gate[k / a.chunks * a.C + c] * p[k * a.C] : p[k * a.C];
  }
  red[sl][lane] = s;
  __syncthreads();
  if (sl || c >= a.C) return;
  for (int k = 1; k < 32; ++k) s += red[k][lane];
  if (blockIdx.y == 0) {
    a.dw_next[c] = s;
    return;
  }
  if (a.dw_post) a.dw_post[c] = scaled || !a.gate ? s : a.gate[c] * s;
  if (a.dgate && !a.row_gate) a.dgate[c] = a.w_post ? a.w_post[c] * s : s;
}

// The gradients of gates that each batch row has for itself.
__global__ void __launch_bounds__(256) residual_gates_kernel(const SumArgs a, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t b = i / a.C;
  const int c = (int)(i - b * a.C);
  float s = 0.f;
  for (int k = 0; k < a.chunks; ++k) s += a.part_h[(b * a.chunks + k) * a.C + c];
  a.dgate[i] = a.w_post ? a.w_post[c] * s : s;
}

constexpr int kMaxC = 8192;
constexpr int kBwdBlocks = 152 * 4;

// Threads of a row, rows of a block.
struct Shape {
  int V, W, threads;
};
Shape shape_of(int64_t C) {
  const int64_t vecs = C / 8;
  Shape s;
  s.V = vecs > 512 ? 2 : 1;
  const int64_t lanes = (vecs + s.V - 1) / s.V;
  s.W = 1;
  while (s.W * 32 < lanes) s.W *= 2;
  s.threads = s.W < 8 ? 256 : s.W * 32;
  return s;
}

struct Units {
  int64_t groups, span;
  int chunks;
};
Units units_of(int64_t B, int64_t T, bool row_gate) {
  Units u;
  u.groups = row_gate ? B : 1;
  u.span = row_gate ? T : B * T;
  int64_t n = kBwdBlocks / u.groups;
  n = n < 1 ? 1 : n;
  u.chunks = (int)(n < u.span ? n : u.span);
  return u;
}

template <typename X, typename Y>
cudaError_t launch_fwd(NormArgs a, cudaStream_t s) {
  const Shape h = shape_of(a.C);
  a.W = h.W;
  const int64_t per = h.threads / 32 / h.W, blocks = (a.rows + per - 1) / per;
  if (h.V == 1) residual_fwd_kernel<X, Y, 1><<<(unsigned)blocks, h.threads, 0, s>>>(a);
  else residual_fwd_kernel<X, Y, 2><<<(unsigned)blocks, h.threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename Y>
cudaError_t launch_bwd(NormArgs a, SumArgs m, cudaStream_t s) {
  const Shape h = shape_of(a.C);
  a.W = h.W;
  const int per = h.threads / 32 / h.W;
  const size_t smem = (size_t)(per - 1) * 2 * a.C * 4;
  const int64_t units = a.groups * a.chunks, blocks = units < kBwdBlocks ? units : kBwdBlocks;
  if (h.V == 1) residual_bwd_kernel<X, Y, 1><<<(unsigned)blocks, h.threads, smem, s>>>(a);
  else residual_bwd_kernel<X, Y, 2><<<(unsigned)blocks, h.threads, smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (m.dw_next || m.dw_post || (m.dgate && !m.row_gate))
    residual_sums_kernel<<<dim3((a.C + 31) / 32, 2), 1024, 0, s>>>(m);
  if (m.dgate && m.row_gate) {
    const int64_t n = a.B * a.C;
    residual_gates_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(m, n);
  }
  return cudaGetLastError();
}

bool rows_aligned(const scan_view4* v, const NormArgs& a, scan_dtype dt) {
  const int64_t n = dt == SCAN_BF16 ? 8 : 4;  // an axis of one element has no stride of its own
  return (uintptr_t)v->ptr % 16 == 0 && (a.B == 1 || v->stride_b % n == 0) && (a.T == 1 || v->stride_t % n == 0);
}

bool given(const scan_view4* v) { return v && v->ptr; }

scan_status norm_common(NormArgs* a, const float* w_post, const float* gate, const float* w_next, int64_t B, int64_t T,
                        int64_t C, int32_t row_gate, float alpha, float eps, double p, uint64_t seed, uint64_t call,
                        const int64_t* rng, scan_dtype sdt, scan_dtype dt) {
  if ((sdt != SCAN_F32 && sdt != SCAN_BF16) || (dt != SCAN_F32 && dt != SCAN_BF16)) return SCAN_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || C < 1 || !(eps >= 0.f) || !(p >= 0. && p <= 1.)) return SCAN_ERR_INVALID_ARG;
  if (!(alpha > -INFINITY && alpha < INFINITY)) return SCAN_ERR_INVALID_ARG;
  if (sdt == SCAN_BF16 && dt == SCAN_F32) return SCAN_ERR_UNSUPPORTED;
  if (C % 8 || C > kMaxC) return SCAN_ERR_UNSUPPORTED;
  if ((double)B * (double)T > 2147483647. || (double)B * (double)C > 1e11) return SCAN_ERR_UNSUPPORTED;  // grids
  if ((uintptr_t)w_post % 16 || (uintptr_t)gate % 16 || (uintptr_t)w_next % 16 || (uintptr_t)rng % 8)
    return SCAN_ERR_ALIGNMENT;
  *a = NormArgs{};
  a->w_post = w_post;
  a->gate = gate;
  a->w_next = w_next;
  a->row_gate = gate && row_gate;
  a->gate_sb = a->row_gate ? C : 0;
  a->B = B;
  a->T = T;
  a->rows = B * T;
  a->C = (int)C;
  a->alpha = alpha;
  a->eps = eps;
  a->inv_C = 1.f / (float)C;
  a->drop = make_drop(p, seed, call, rng);
  return SCAN_OK;
}

}  // namespace
}  // namespace scan

using namespace scan;

extern "C" {

size_t residual_norm_workspace_bytes(int64_t B, int64_t T, int64_t C, int32_t row_gate) {
  if (B < 0 || T < 0 || C < 1 || C % 8 || C > kMaxC) return 0;
  if (B == 0 || T == 0) return 16;
  if ((double)B * (double)T > 2147483647.) return 0;
  const Units u = units_of(B, T, row_gate != 0);
  return (size_t)(u.groups * u.chunks) * 2 * (size_t)C * 4;
}

scan_status residual_norm_fwd(const scan_view4* x, const scan_view4* y, const float* post_weight, const float* gate,
                              const float* next_weight, const scan_view4* x_out, const scan_view4* n, int64_t B,
                              int64_t T, int64_t C, int32_t row_gate, float alpha, float eps, double p,
                              uint64_t seed, uint64_t call, const int64_t* rng, scan_dtype stream_dt, scan_dtype dt,
                              cudaStream_t stream) {
  NormArgs a;
  const scan_status st = norm_common(&a, post_weight, gate, next_weight, B, T, C, row_gate, alpha, eps, p, seed, call,
                                     rng, stream_dt, dt);
  if (st != SCAN_OK) return st;
  if (!y && (post_weight || gate || !next_weight || alpha != 1.f || p != 0.)) return SCAN_ERR_INVALID_ARG;
  if (a.rows == 0) return SCAN_OK;
  if (!given(x) || (y && (!y->ptr || !given(x_out))) || (next_weight && !given(n))) return SCAN_ERR_INVALID_ARG;
  if (!rows_aligned(x, a, stream_dt) || (y && (!rows_aligned(y, a, dt) || !rows_aligned(x_out, a, stream_dt))) ||
      (next_weight && !rows_aligned(n, a, dt)))
    return SCAN_ERR_ALIGNMENT;
  a.x = x->ptr, a.x_sb = x->stride_b, a.x_st = x->stride_t;
  if (y) {
    a.y = y->ptr, a.y_sb = y->stride_b, a.y_st = y->stride_t;
    a.xo = x_out->ptr, a.xo_sb = x_out->stride_b, a.xo_st = x_out->stride_t;
  }
  if (next_weight) a.n = n->ptr, a.n_sb = n->stride_b, a.n_st = n->stride_t;
  const cudaError_t e = stream_dt == SCAN_BF16 ? launch_fwd<__nv_bfloat16, __nv_bfloat16>(a, stream)
                        : dt == SCAN_BF16      ? launch_fwd<float, __nv_bfloat16>(a, stream)
                                               : launch_fwd<float, float>(a, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status residual_norm_bwd(const scan_view4* x_out, const scan_view4* y, const scan_view4* dx_out,
                              const scan_view4* dn, const float* post_weight, const float* gate,
                              const float* next_weight, const scan_view4* dx, const scan_view4* dy,
                              float* dpost_weight, float* dgate, float* dnext_weight, int64_t B, int64_t T, int64_t C,
                              int32_t row_gate, float alpha, float eps, double p, uint64_t seed, uint64_t call,
                              const int64_t* rng, scan_dtype stream_dt, scan_dtype dt, void* workspace,
                              size_t workspace_bytes, cudaStream_t stream) {
  NormArgs a;
  const scan_status st = norm_common(&a, post_weight, gate, next_weight, B, T, C, row_gate, alpha, eps, p, seed, call,
                                     rng, stream_dt, dt);
  if (st != SCAN_OK) return st;
  if (!y && (post_weight || gate || !next_weight || alpha != 1.f || p != 0.)) return SCAN_ERR_INVALID_ARG;
  if ((dpost_weight && !post_weight) || (dgate && !gate) || (dnext_weight && !next_weight)) return SCAN_ERR_INVALID_ARG;
  if (a.rows == 0) {  // no rows: the weights' gradients are 0
    cudaError_t e = cudaSuccess;
    if (dpost_weight) e = launch_fill_zero(dpost_weight, C, stream);
    if (e == cudaSuccess && dgate && (a.row_gate ? B : 1) > 0)
      e = launch_fill_zero(dgate, (a.row_gate ? B : 1) * C, stream);
    if (e == cudaSuccess && dnext_weight) e = launch_fill_zero(dnext_weight, C, stream);
    return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
  }
  if (!given(dx) || (y && (!y->ptr || !given(dy))) || (next_weight && (!given(x_out) || !given(dn))) ||
      (!next_weight && !given(dx_out)))
    return SCAN_ERR_INVALID_ARG;
  if (!rows_aligned(dx, a, stream_dt) || (given(dx_out) && !rows_aligned(dx_out, a, stream_dt)) ||
      (y && (!rows_aligned(y, a, dt) || !rows_aligned(dy, a, dt))) ||
      (next_weight && (!rows_aligned(x_out, a, stream_dt) || !rows_aligned(dn, a, dt))))
    return SCAN_ERR_ALIGNMENT;
  if (!workspace || (uintptr_t)workspace % 16 ||
      workspace_bytes < residual_norm_workspace_bytes(B, T, C, a.row_gate))
    return SCAN_ERR_WORKSPACE;
  if (next_weight) {
    a.x = x_out->ptr, a.x_sb = x_out->stride_b, a.x_st = x_out->stride_t;
    a.dn = dn->ptr, a.n_sb = dn->stride_b, a.n_st = dn->stride_t;
  }
  if (given(dx_out)) a.dxo = dx_out->ptr, a.xo_sb = dx_out->stride_b, a.xo_st = dx_out->stride_t;
  a.dx = dx->ptr, a.dx_sb = dx->stride_b, a.dx_st = dx->stride_t;
  if (y) {
    a.y = y->ptr, a.y_sb = y->stride_b, a.y_st = y->stride_t;
    a.dy = dy->ptr, a.dy_sb = dy->stride_b, a.dy_st = dy->stride_t;
  }
  const Units u = units_of(B, T, a.row_gate);
  a.groups = u.groups;
  a.span = u.span;
  a.chunks = u.chunks;
  a.part_h = static_cast<float*>(workspace);
  a.part_n = a.part_h + u.groups * u.chunks * C;
  const SumArgs m{a.part_h, a.part_n, post_weight, gate, dpost_weight, dgate, dnext_weight, u.groups * u.chunks,
                  a.C, u.chunks, a.row_gate};
  const cudaError_t e = stream_dt == SCAN_BF16 ? launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, m, stream)
                        : dt == SCAN_BF16      ? launch_bwd<float, __nv_bfloat16>(a, m, stream)
                                               : launch_bwd<float, float>(a, m, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // extern "C"
