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
// cover it, one, two or four times eight elements a thread (fwd_shape, bwd_shape), so that no
// row is read twice. Sums are shuffles and an exchange through shared memory: one a norm
// forward, one of six sums backward.
// 8 x 4096 rows of 2048, the stream in fp32, y in bf16, dropout: forward 134 us (6.0 TB/s),
// backward 195 us and the sums 11 us (6.2 TB/s during the walk).
#include "scan_mixer.h"
#include "scan_philox.cuh"
#include "scan_tc.cuh"

namespace scan {
namespace {

using tc::add2;
using tc::fma2;
using tc::mul2;

struct NormArgs {
  const void *x, *y, *dxo, *dn;  // forward: x, y; backward: x', y, dx', dn
  void *xo, *n, *dx, *dy;
  int64_t x_sb, x_st, y_sb, y_st, xo_sb, xo_st, n_sb, n_st;  // (backward: xo = dx', n = dn)
  int64_t dx_sb, dx_st, dy_sb, dy_st;
  const float *w_post, *gate, *w_next;  // nullable
  int64_t gate_sb;                      // C where each batch row has a gate, else 0
  int64_t B, T, rows;
  int C, W;          // W: warps a row
  int wide;          // rows of the stream and of gradients are on 32 bytes
  float alpha, eps, inv_C;
  Drop drop;
  // backward
  WsHeader* hdr;
  float *part_h, *part_n;  // [units][C]
  int64_t groups, span;    // rows that share a gate: `groups` runs of `span` rows
  int chunks;              // units a group
  int row_gate;
};

__device__ __forceinline__ float4 shared16(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}

// Eight elements of a row, in memory and as numbers.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, bool wide) {  // wide: p is on 32 bytes
    if (wide) {
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                   : "l"(p));
    } else {
      a = *reinterpret_cast<const float4*>(p);
      b = *(reinterpret_cast<const float4*>(p) + 1);
    }
  }
  __device__ __forceinline__ void clear() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void take(uint32_t at, uint32_t apart) {  // pieces in shared memory
    a = shared16(at);
    b = shared16(at + apart);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const float2 (&v)[4]) {
    a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    b = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
  __device__ __forceinline__ void store(float* p, bool wide) const {
    if (wide) {
      asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(a.x), "f"(a.y), "f"(a.z), "f"(a.w),
                   "f"(b.x), "f"(b.y), "f"(b.z), "f"(b.w), "l"(p)
                   : "memory");
    } else {
      *reinterpret_cast<float4*>(p) = a;
      *(reinterpret_cast<float4*>(p) + 1) = b;
    }
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void clear() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void take(uint32_t at, uint32_t) {
    const float4 v = shared16(at);
    a = make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void set(const float2 (&v)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, bool) const { *reinterpret_cast<uint4*>(p) = a; }
};

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Weights of eight columns, ones where there are none.
__device__ __forceinline__ void weights(const float* w, int c, bool on, float2 (&v)[4]) {
  Eight<float> e;
  if (w && on) {
    e.load(w + c, false);
    e.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = both(1.f);
  }
}

// Sums of up to four numbers over the W warps of a row, in warp order, for all its
// threads. `red`: one slot a warp of the block; every thread of the block comes here.
template <int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float4* red, int W) {
#pragma unroll
  for (int d = 16; d; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], d);
  if (W == 1) return;
  const int warp = threadIdx.x / 32, first = warp / W * W;
  if (threadIdx.x % 32 == 0) red[warp] = make_float4(s[0], N > 1 ? s[N > 1 ? 1 : 0] : 0.f, N > 2 ? s[N > 2 ? 2 : 0] : 0.f, 0.f);
  __syncthreads();
  float4 t = red[first];
  for (int w = 1; w < W; ++w) {
    const float4 o = red[first + w];
    t.x += o.x, t.y += o.y, t.z += o.z;
  }
  s[0] = t.x;
  if (N > 1) s[N > 1 ? 1 : 0] = t.y;
  if (N > 2) s[N > 2 ? 2 : 0] = t.z;
}

// V: vectors of eight elements a thread.
template <typename X, typename Y, int V>
__global__ void __launch_bounds__(512) residual_fwd_kernel(const NormArgs a) {
  __shared__ float4 red[2][16];
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
      ex[v].load(x + c, a.wide);
      if (a.y) ey[v].load(y + c, a.wide);
    }
  }
  if (a.y) {
    uint64_t seed, call;
    a.drop.read(&seed, &call);
    float r = 1.f;
    if (a.w_post) {
      float2 sq = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float2 f[4];
        ey[v].get(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = fma2(f[i], f[i], sq);
      }
      float s[1] = {sq.x + sq.y};
      row_sums(s, red[0], a.W);
      r = rsqrtf(fmaf(s[0], a.inv_C, a.eps));
    }
    X* const xo = static_cast<X*>(a.xo) + b * a.xo_sb + t * a.xo_st;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * (lane + v * 32 * a.W);
      const bool on = live && c < a.C;
      float2 f[4], g[4], w[4];
      ey[v].get(f);
      weights(a.w_post, c, on, w);
      weights(a.gate ? a.gate + b * a.gate_sb : nullptr, c, on, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], both(r)), mul2(w[i], g[i]));
      if (a.drop.limit) drop8(f, a.drop, (uint64_t)(row * (a.C / 8) + c / 8), call, seed);
      ex[v].get(g);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = fma2(both(a.alpha), g[i], f[i]);
      ex[v].set(f);
      if (on) ex[v].store(xo + c, a.wide);
    }
  }
  if (!a.w_next) return;
  float2 sq = both(0.f);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float2 f[4];
    ex[v].get(f);
    if (8 * (lane + v * 32 * a.W) < a.C)
#pragma unroll
      for (int i = 0; i < 4; ++i) sq = fma2(f[i], f[i], sq);
  }
  float s[1] = {sq.x + sq.y};
  row_sums(s, red[1], a.W);
  const float q = rsqrtf(fmaf(s[0], a.inv_C, a.eps));
  Y* const n = static_cast<Y*>(a.n) + b * a.n_sb + t * a.n_st;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * (lane + v * 32 * a.W);
    const bool on = live && c < a.C;
    float2 f[4], w[4];
    ex[v].get(f);
    weights(a.w_next, c, on, w);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mul2(mul2(f[i], both(q)), w[i]);
    Eight<Y> e;
    e.set(f);
    if (on) e.store(n + c, a.wide);
  }
}

// A run of a row to shared memory; `bar` counts its bytes.
__device__ __forceinline__ void copy_run(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
               "l"(from), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void keep16(uint32_t at, float2 a, float2 b) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y) : "memory");
}

// Sums of six numbers over the W warps of a row, for all its threads: a lane keeps half
// of the numbers at each of three exchanges (16, 8 and 4 lanes away), so that seven
// exchanges serve all; then the warps' in order. `red`: a slot a warp of the block.
__device__ __forceinline__ void six_sums(float (&s)[6], float4 (*red)[2], int W) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, first = warp / W * W;
  float v[4] = {s[0], s[1], s[2], s[3]};
  {
    const bool up = lane & 16;
    const float u[4] = {s[4], s[5], 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (up ? u[i] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : u[i], 16);
  }
  {
    const bool up = lane & 8;
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = (up ? v[i + 2] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 2], 8);
  }
  {
    const bool up = lane & 4;
    v[0] = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 4);
  }
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
  v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
  if (lane % 4 == 0) reinterpret_cast<float*>(red[warp])[lane / 4] = v[0];
  if (W == 1) __syncwarp();
  else __syncthreads();
  float4 a = red[first][0], b = red[first][1];
  for (int w = 1; w < W; ++w) {
    const float4 c = red[first + w][0], d = red[first + w][1];
    a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w, b.x += d.x, b.y += d.y;
  }
  s[0] = a.x, s[1] = a.y, s[2] = a.z, s[3] = a.w, s[4] = b.x, s[5] = b.y;
}

// A block walks units: every chunks-th row of those that share a gate (so that blocks at
// work are at neighbouring rows), its column sums in registers, left in the workspace and
// added in order by the kernel below. A row's operands are copied to shared memory as
// whole runs, AHEAD rows ahead, by one thread of its own; the unit's weights lie there as
// well. Where the rows to come begin is worked out by six threads, one an operand, which
// leave it in shared memory: six walks in every thread took 30 registers. Copies by the
// threads themselves, 16 bytes each, moved every sector of the fp32 operands twice.
template <typename X, typename Y, int V, int AHEAD>
__global__ void __launch_bounds__(V == 4 ? 256 : 128, V == 4 ? 1 : 3) residual_bwd_kernel(const NormArgs a) {
  constexpr int NS = AHEAD + 1;  // 1, 2 or 4
  __shared__ float4 red[2][8][2];
  __shared__ char* begins[8][8][6];  // a slot a row of the block
  __shared__ uint64_t bars[8][NS];
  __shared__ uint32_t expired;
  // [NS][rows a block] of x', dx', y, dn; the weights' pieces [4 V][threads a row]; then the
  // fold: [rows a block - 1][2][C]
  extern __shared__ float4 ring[];
  const int per = blockDim.x / 32 / a.W, lane = threadIdx.x % (32 * a.W), mine = threadIdx.x / (32 * a.W);
  const uint32_t run_x = a.C * sizeof(X), run_y = a.C * sizeof(Y), run = 2 * (run_x + run_y);
  const uint32_t apart = 32 * a.W * 16;  // bytes between a thread's pieces of the weights
  const uint32_t rows_at = tc::smem_addr(ring), own_w = rows_at + NS * per * run + lane * 16;
  const uint32_t bar0 = tc::smem_addr(&bars[mine][0]);
  const tc::Stop stop{&expired, a.hdr};
  float* const fold = reinterpret_cast<float*>(ring);
  const int64_t units = a.groups * a.chunks;
  asm volatile("griddepcontrol.launch_dependents;");  // the sums' blocks come beside this one's
  uint64_t seed, call;
  a.drop.read(&seed, &call);
  const int c0 = 8 * lane, apart_c = 8 * 32 * a.W;  // a thread's first column, and from vector to vector
  if (threadIdx.x == 0) expired = 0;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) tc::bar_init(bar0 + 8 * i, 1);
    tc::bar_init_fence();
  }
  uint32_t turn = 0;  // rows walked before this unit
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t grp = unit / a.chunks, ch = unit - grp * a.chunks;
    const int64_t beg = grp * a.span + ch * per, end = (grp + 1) * a.span, step = (int64_t)a.chunks * per;
    const int64_t on_b = step / a.T, on_t = step - on_b * a.T;
    const float* const gate = a.gate ? a.gate + (a.row_gate ? grp * a.gate_sb : 0) : nullptr;
    float2 h[V][4], dw[V][4];
    tc::fence_async();  // (the fold's writes, before copies to the same place)
    __syncthreads();    // the last unit's rows are done
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = c0 + v * apart_c;
      float2 wn[4], wu[4];  // next_weight; post_weight times gate
      weights(a.w_next, c, c < a.C, wn);
      weights(a.w_post, c, c < a.C, wu);
      weights(gate, c, c < a.C, h[v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wu[i] = mul2(wu[i], h[v][i]);
        h[v][i] = dw[v][i] = both(0.f);
      }
      if (mine == 0) {
        keep16(own_w + (4 * v) * apart, wn[0], wn[1]);
        keep16(own_w + (4 * v + 1) * apart, wn[2], wn[3]);
        keep16(own_w + (4 * v + 2) * apart, wu[0], wu[1]);
        keep16(own_w + (4 * v + 3) * apart, wu[2], wu[3]);
      }
    }
    // x', dx', y, dn, dx, dy of the rows to come, until one row after their own
    char* next = nullptr;
    int64_t on = 0, wrap = 0, at_t = 0;
    if (lane < 6) {
      const int64_t b = (beg + mine) / a.T;
      at_t = beg + mine - b * a.T;
      const bool x = lane == 0 || lane == 1 || lane == 4;
      const int64_t sb = lane == 0 ? a.x_sb : lane == 1 ? a.xo_sb : lane == 2 ? a.y_sb : lane == 3 ? a.n_sb : lane == 4 ? a.dx_sb : a.dy_sb;
      const int64_t st = lane == 0 ? a.x_st : lane == 1 ? a.xo_st : lane == 2 ? a.y_st : lane == 3 ? a.n_st : lane == 4 ? a.dx_st : a.dy_st;
      const void* const base = lane == 0 ? a.x : lane == 1 ? a.dxo : lane == 2 ? a.y : lane == 3 ? a.dn : lane == 4 ? a.dx : a.dy;
      const int64_t size = x ? sizeof(X) : sizeof(Y);
      next = static_cast<char*>(const_cast<void*>(base)) + (b * sb + at_t * st) * size;
      on = (on_b * sb + on_t * st) * size;
      wrap = (sb - a.T * st) * size;
    }
    char* const* const mine_at = &begins[mine][0][0];
    const auto begin_of = [&](int i) {
      if (lane < 6) {
        begins[mine][i & 7][lane] = next;
        next += on;
        at_t += on_t;
        if (at_t >= a.T) at_t -= a.T, next += wrap;
      }
    };
    for (int i = 0; i <= AHEAD; ++i) begin_of(i);
    __syncthreads();
    // row r0 of the block's next ones, this thread's among them: the i-th of the unit
    const auto copy = [&](int64_t r0, int i) {
      if (lane == 0 && r0 < end) {
        const uint32_t slot = (turn + i) % NS, bar = bar0 + 8 * slot;
        if (r0 + mine < end) {
          const uint32_t to = rows_at + (slot * per + mine) * run;
          char* const* const from = mine_at + (i & 7) * 6;
          tc::bar_expect(bar, (a.x ? run_x + run_y : 0) + (a.dxo ? run_x : 0) + (a.y ? run_y : 0));
          if (a.x) copy_run(to, from[0], run_x, bar);
          if (a.dxo) copy_run(to + run_x, from[1], run_x, bar);
          if (a.y) copy_run(to + 2 * run_x, from[2], run_y, bar);
          if (a.x) copy_run(to + 2 * run_x + run_y, from[3], run_y, bar);
        } else {
          tc::bar_arrive(bar);
        }
      }
    };
    int odd = 0, count = 0;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) copy(beg + i * step, i);
    for (int64_t r0 = beg; r0 < end; r0 += step, ++count) {
      const int64_t row = r0 + mine;
      const bool live = row < end;
      begin_of(count + AHEAD + 1);
      copy(r0 + AHEAD * step, count + AHEAD);
      const uint32_t slot = (turn + count) % NS, at0 = rows_at + (slot * per + mine) * run;
      tc::bar_wait(bar0 + 8 * slot, (turn + count) / NS & 1, stop);
      // x', dx', y, dn; zeros where there is nothing
      Eight<X> ex[V], eg[V];
      Eight<Y> ey[V], en[V];
      uint32_t keep[V];  // a bit an element
      float2 sum[6];     // y y; x' x'; e x'; and of d = post_weight gate y / (1 - p) where kept: d dx', d e, d x'
#pragma unroll
      for (int i = 0; i < 6; ++i) sum[i] = both(0.f);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * apart_c;
        const uint32_t at_x = at0 + c * sizeof(X), at_y = at0 + 2 * run_x + c * sizeof(Y);
        const bool here = live && c < a.C;
        ex[v].clear(), eg[v].clear(), ey[v].clear(), en[v].clear();
        if (here && a.x) ex[v].take(at_x, 16), en[v].take(at_y + run_y, 16);
        if (here && a.dxo) eg[v].take(at_x + run_x, 16);
        if (here && a.y) ey[v].take(at_y, 16);
        float2 x[4], g[4], y[4], e[4], w[4];
        ex[v].get(x);
        en[v].get(e);
        Eight<float> held;
        held.take(own_w + 4 * v * apart, apart);
        held.get(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = mul2(e[i], w[i]);
          sum[1] = fma2(x[i], x[i], sum[1]);
          sum[2] = fma2(e[i], x[i], sum[2]);
        }
        keep[v] = 0xffu;
        if (a.y) {
          ey[v].get(y);
          eg[v].get(g);
          held.take(own_w + (4 * v + 2) * apart, apart);
          held.get(w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[0] = fma2(y[i], y[i], sum[0]);
            w[i] = mul2(w[i], y[i]);
          }
          if (a.drop.limit) {
            keep[v] = kept8(a.drop, (uint64_t)(row * (a.C / 8) + c / 8), call, seed);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              w[i].x = keep[v] & 1u << 2 * i ? w[i].x * a.drop.scale : 0.f;
              w[i].y = keep[v] & 2u << 2 * i ? w[i].y * a.drop.scale : 0.f;
              g[i].x = keep[v] & 1u << 2 * i ? g[i].x : 0.f;
              g[i].y = keep[v] & 2u << 2 * i ? g[i].y : 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[3] = fma2(w[i], g[i], sum[3]);
            sum[4] = fma2(w[i], e[i], sum[4]);
            sum[5] = fma2(w[i], x[i], sum[5]);
          }
        }
      }
      float s[6];
#pragma unroll
      for (int i = 0; i < 6; ++i) s[i] = sum[i].x + sum[i].y;
      six_sums(s, red[odd], a.W);
      odd ^= 1;
      // a row that is not there is zeros and adds nothing, also where eps is 0
      const float r = !a.w_post ? 1.f : live ? rsqrtf(fmaf(s[0], a.inv_C, a.eps)) : 0.f;
      const float q = live && a.w_next ? rsqrtf(fmaf(s[1], a.inv_C, a.eps)) : 0.f;
      const float mean = s[2] * a.inv_C * q;                                        // of e x' q
      // of f y r, f = post_weight gate u: G is linear in what is known by now
      const float mean2 = a.w_post ? fmaf(q, fmaf(-q * mean, s[5], s[4]), s[3]) * a.inv_C * r : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * apart_c;
        const bool here = live && c < a.C;
        float2 x[4], e[4], g[4], w[4];
        ex[v].get(x);
        en[v].get(e);
        eg[v].get(g);
        Eight<float> held;
        held.take(own_w + 4 * v * apart, apart);
        held.get(w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = mul2(x[i], both(q));
          dw[v][i] = fma2(e[i], x[i], dw[v][i]);
          g[i] = fma2(both(q), fma2(x[i], both(-mean), mul2(e[i], w[i])), g[i]);
          e[i] = mul2(g[i], both(a.alpha));
        }
        Eight<X> out;
        out.set(e);
        if (here) out.store(reinterpret_cast<X*>(mine_at[(count & 7) * 6 + 4]) + c, a.wide);
        if (a.y) {
          if (a.drop.limit)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              g[i].x = keep[v] & 1u << 2 * i ? g[i].x * a.drop.scale : 0.f;
              g[i].y = keep[v] & 2u << 2 * i ? g[i].y * a.drop.scale : 0.f;
            }
          ey[v].get(x);
          if (a.drop.limit && !a.w_post)  // what was dropped may have been anything (a norm would have taken it in)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i].x = keep[v] & 1u << 2 * i ? x[i].x : 0.f;
              x[i].y = keep[v] & 2u << 2 * i ? x[i].y : 0.f;
            }
          held.take(own_w + (4 * v + 2) * apart, apart);
          held.get(w);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = mul2(x[i], both(r));
            h[v][i] = fma2(g[i], x[i], h[v][i]);
            g[i] = mul2(both(r), fma2(x[i], both(-mean2), mul2(g[i], w[i])));
          }
          Eight<Y> back;
          back.set(g);
          if (here) back.store(reinterpret_cast<Y*>(mine_at[(count & 7) * 6 + 5]) + c, a.wide);
        }
      }
    }
    turn += count;
    // the block's rows, in order
    if (per > 1) {
      __syncthreads();
      if (mine > 0)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = c0 + v * apart_c;
          if (c < a.C)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              *reinterpret_cast<float2*>(fold + ((mine - 1) * 2) * a.C + c + 2 * i) = h[v][i];
              *reinterpret_cast<float2*>(fold + ((mine - 1) * 2 + 1) * a.C + c + 2 * i) = dw[v][i];
            }
        }
      __syncthreads();
    }
    if (mine == 0)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = c0 + v * apart_c;
        if (c >= a.C) continue;
        for (int k = 0; k < per - 1; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[v][i] = add2(h[v][i], *reinterpret_cast<const float2*>(fold + (k * 2) * a.C + c + 2 * i));
            dw[v][i] = add2(dw[v][i], *reinterpret_cast<const float2*>(fold + (k * 2 + 1) * a.C + c + 2 * i));
          }
        Eight<float> e;
        e.set(h[v]);
        e.store(a.part_h + unit * a.C + c, false);
        e.set(dw[v]);
        e.store(a.part_n + unit * a.C + c, false);
      }
    if (per > 1) __syncthreads();
  }
  tc::linger(stop);
}

struct SumArgs {
  const float *part_h, *part_n, *w_post, *gate;
  float *dw_post, *dgate, *dw_next;
  int64_t units;
  int C, chunks, row_gate;
};

// Columns of the partial sums: 32 lanes of columns by 32 slices of units, the slices
// then added in order. blockIdx.y 0: dw_next; 1: dw_post and a shared gate's gradient;
// 2 ..: the gradients of gates that each batch row has for itself.
__global__ void __launch_bounds__(1024) residual_sums_kernel(const SumArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the walk's end
  const int lane = threadIdx.x % 32, c = blockIdx.x * 32 + lane, sl = threadIdx.x / 32, y = blockIdx.y;
  if (y == 0 ? !a.dw_next : y == 1 ? !a.dw_post && (!a.dgate || a.row_gate) : !a.dgate) return;
  __shared__ float red[32][33];
  const float* const p = (y ? a.part_h : a.part_n) + c;
  const bool scaled = y == 1 && a.row_gate;
  const int first = y > 1 ? (y - 2) * a.chunks : 0, last = y > 1 ? first + a.chunks : (int)a.units;
  float s = 0.f;
  if (c < a.C) {
#pragma unroll 16
    for (int k = first + sl; k < last; k += 32)
      s += scaled ? a.gate[(int64_t)(k / a.chunks) * a.C + c] * p[(int64_t)k * a.C] : p[(int64_t)k * a.C];
  }
  red[sl][lane] = s;
  __syncthreads();
  if (sl || c >= a.C) return;
  for (int k = 1; k < 32; ++k) s += red[k][lane];
  if (y == 0) {
    a.dw_next[c] = s;
  } else if (y > 1) {
    a.dgate[(int64_t)(y - 2) * a.C + c] = a.w_post ? a.w_post[c] * s : s;
  } else {
    if (a.dw_post) a.dw_post[c] = scaled || !a.gate ? s : a.gate[c] * s;
    if (a.dgate && !a.row_gate) a.dgate[c] = a.w_post ? a.w_post[c] * s : s;
  }
}

// The gradients of gates of more batch rows than there are blocks, whose sums are whole.
__global__ void __launch_bounds__(256) residual_gates_kernel(const SumArgs a, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) a.dgate[i] = a.w_post ? a.w_post[i % a.C] * a.part_h[i] : a.part_h[i];
}

constexpr int kMaxC = 8192;
constexpr int kSms = 152;
constexpr int kMostBlocks = 3 * kSms;  // of the backward's walk

// Vectors of eight elements a thread, warps a row, threads a block.
struct Shape {
  int V, W, threads;
};
Shape shape_with(int C, int V, int threads) {
  Shape s{V, 1, threads};
  while (s.W * 32 * V * 8 < C) s.W *= 2;
  if (s.W * 32 > threads) s.threads = s.W * 32;
  return s;
}
// Forward: four vectors a thread and small blocks, so that much is on its way with little
// to wait for: 8 x 4096 rows of 2048 in us, by vectors a thread, blocks of 64 / 256
// threads: 202 / 202 (1), 147 / 157 (2), 143 / 171 (4), 146 / 144 (8). Few rows are
// spread over more threads instead.
Shape fwd_shape(int C, int64_t rows) {
  if (C <= 256 || (rows < 8 * kSms && C <= 4096)) return shape_with(C, 1, 64);
  return shape_with(C, C <= 512 ? 2 : 4, 64);
}
// Backward: two vectors a thread where 128 threads hold a row of them: 8 x 4096 rows of
// 2048 in us, launches included: 231 with two vectors and three blocks an SM (registers
// held to 168; for four they would spill), 277 with two blocks, 342 with four vectors.
Shape bwd_shape(int C) { return shape_with(C, C <= 256 ? 1 : C <= 2048 ? 2 : 4, 128); }

struct Units {
  int64_t groups, span;
  int chunks;
};
Units units_of(int64_t B, int64_t T, bool row_gate, int blocks) {
  Units u;
  u.groups = row_gate ? B : 1;
  u.span = row_gate ? T : B * T;
  int64_t n = blocks / u.groups;
  n = n < 1 ? 1 : n;
  u.chunks = (int)(n < u.span ? n : u.span);
  return u;
}

// The backward's copies run three rows ahead or one, or not at all, as shared memory
// holds them; and how many blocks an SM then holds. Blocks come before depth (the rows
// above: 231 us one row ahead in three blocks, 290 not ahead, 438 three ahead in two).
struct Ring {
  int ahead, per_sm;
  size_t bytes;
};
Ring ring_of(const Shape& h, int C, int bytes) {
  const size_t row = (size_t)(h.threads / 32 / h.W) * C * bytes, held = (size_t)h.V * 4 * h.W * 32 * 16;
  const size_t sm = (size_t)221 << 10, third = (size_t)70 << 10, fixed = 5 << 10;  // fixed: what a block has besides
  Ring r;
  r.ahead = 4 * row + held <= third ? 3 : 2 * row + held <= sm ? 1 : 0;
  r.bytes = (r.ahead + 1) * row + held;
  const int fit = (int)(((size_t)228 << 10) / (r.bytes + fixed)), regs = h.V < 4 ? 3 : h.threads <= 128 ? 2 : 1;
  r.per_sm = fit < 1 ? 1 : fit < regs ? fit : regs;
  return r;
}
int bytes_of(scan_dtype stream_dt, scan_dtype dt) {  // of x', dx', y and dn, an element of each
  return 2 * (stream_dt == SCAN_BF16 ? 2 : 4) + 2 * (dt == SCAN_BF16 ? 2 : 4);
}

template <typename X, typename Y>
cudaError_t launch_fwd(NormArgs a, cudaStream_t s) {
  const Shape h = fwd_shape(a.C, a.rows);
  a.W = h.W;
  const int64_t per = h.threads / 32 / h.W, blocks = (a.rows + per - 1) / per;
  if (h.V == 1) residual_fwd_kernel<X, Y, 1><<<(unsigned)blocks, h.threads, 0, s>>>(a);
  else if (h.V == 2) residual_fwd_kernel<X, Y, 2><<<(unsigned)blocks, h.threads, 0, s>>>(a);
  else residual_fwd_kernel<X, Y, 4><<<(unsigned)blocks, h.threads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename X, typename Y, int V, int AHEAD>
cudaError_t launch_walk(const NormArgs& a, const Shape& h, const Ring& r, cudaStream_t s) {
  const size_t fold = (size_t)(h.threads / 32 / h.W - 1) * 2 * a.C * 4, smem = r.bytes > fold ? r.bytes : fold;
  const cudaError_t e =
      cudaFuncSetAttribute(residual_bwd_kernel<X, Y, V, AHEAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t units = a.groups * a.chunks, blocks = units < r.per_sm * kSms ? units : r.per_sm * kSms;
  residual_bwd_kernel<X, Y, V, AHEAD><<<(unsigned)blocks, h.threads, smem, s>>>(a);
  return cudaGetLastError();
}
template <typename X, typename Y, int V>
cudaError_t launch_walk(const NormArgs& a, const Shape& h, const Ring& r, cudaStream_t s) {
  if (r.ahead == 3) return launch_walk<X, Y, V, 3>(a, h, r, s);
  if (r.ahead == 1) return launch_walk<X, Y, V, 1>(a, h, r, s);
  return launch_walk<X, Y, V, 0>(a, h, r, s);
}

template <typename X, typename Y>
cudaError_t launch_bwd(NormArgs a, SumArgs m, const Shape& h, const Ring& r, cudaStream_t s) {
  a.W = h.W;
  cudaError_t e = h.V == 1   ? launch_walk<X, Y, 1>(a, h, r, s)
                  : h.V == 2 ? launch_walk<X, Y, 2>(a, h, r, s)
                             : launch_walk<X, Y, 4>(a, h, r, s);
  if (e != cudaSuccess) return e;
  const bool gates = m.dgate && m.row_gate, single = gates && m.chunks == 1;
  if (m.dw_next || m.dw_post || (m.dgate && !single)) {
    // launched while the walk runs, whose end it waits for itself
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.C + 31) / 32, gates && !single ? (unsigned)(2 + a.B) : 2u);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, residual_sums_kernel, m);
    if (e != cudaSuccess) return e;
  }
  if (single) residual_gates_kernel<<<(unsigned)((a.B * a.C + 255) / 256), 256, 0, s>>>(m, a.B * a.C);
  return cudaGetLastError();
}

bool rows_aligned(const scan_view4* v, const NormArgs& a, scan_dtype dt) {
  const int64_t n = dt == SCAN_BF16 ? 8 : 4;  // an axis of one element has no stride of its own
  return (uintptr_t)v->ptr % 16 == 0 && (a.B == 1 || v->stride_b % n == 0) && (a.T == 1 || v->stride_t % n == 0);
}

// fp32 rows on 32 bytes (bf16 ones take 16-byte pieces anyway).
bool rows_wide(const scan_view4* v, const NormArgs& a, scan_dtype dt) {
  return !v || !v->ptr || dt == SCAN_BF16 ||
         ((uintptr_t)v->ptr % 32 == 0 && (a.B == 1 || v->stride_b % 8 == 0) && (a.T == 1 || v->stride_t % 8 == 0));
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
  if (B == 0 || T == 0) return kWsHeaderBytes;
  if ((double)B * (double)T > 2147483647.) return 0;
  const Units u = units_of(B, T, row_gate != 0, kMostBlocks);
  return kWsHeaderBytes + (size_t)(u.groups * u.chunks) * 2 * (size_t)C * 4;
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
  a.wide = rows_wide(x, a, stream_dt) && rows_wide(y, a, dt) && (!y || rows_wide(x_out, a, stream_dt)) &&
           (!next_weight || rows_wide(n, a, dt));
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
  a.wide = rows_wide(dx, a, stream_dt) && rows_wide(dx_out, a, stream_dt) && rows_wide(y, a, dt) &&
           (!y || rows_wide(dy, a, dt)) && (!next_weight || (rows_wide(x_out, a, stream_dt) && rows_wide(dn, a, dt)));
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
  const Shape h = bwd_shape(a.C);
  const Ring r = ring_of(h, a.C, bytes_of(stream_dt, dt));
  const Units u = units_of(B, T, a.row_gate, r.per_sm * kSms);
  a.groups = u.groups;
  a.span = u.span;
  a.chunks = u.chunks;
  a.hdr = static_cast<WsHeader*>(workspace);
  a.part_h = reinterpret_cast<float*>(static_cast<char*>(workspace) + kWsHeaderBytes);
  a.part_n = a.part_h + u.groups * u.chunks * C;
  const SumArgs m{a.part_h, a.part_n, post_weight, gate, dpost_weight, dgate, dnext_weight, u.groups * u.chunks,
                  a.C, u.chunks, a.row_gate};
  const cudaError_t e = stream_dt == SCAN_BF16 ? launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, m, h, r, stream)
                        : dt == SCAN_BF16      ? launch_bwd<float, __nv_bfloat16>(a, m, h, r, stream)
                                               : launch_bwd<float, float>(a, m, h, r, stream);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // extern "C"
