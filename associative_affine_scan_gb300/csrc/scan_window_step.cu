// scan_window_step.cu -- sliding-window attention of one token a request over its
// ring of cached keys and values (bf16 caches).
//
// Bound by DRAM: each cached row is read once for the query heads that share it
// (4 G multiply-adds a byte pair at most). A warp takes 16 keys at a time, by 16-byte
// loads; the next keys' are issued when these have been used and the next values' when
// these have, so 4 to 8 KB a warp are always on their way. Two sets of m16n8k16
// products: scores of up to 16 query heads (the rows) by 16 keys, and weights by V.
// The sums' index order is free, so each fragment is what a thread loaded 16 bytes
// of: the scores' index runs over the D elements in the order of the four lanes'
// pieces, and the columns of the output are the elements in the order 8 n + j.
// Fragments of V pair two keys' elements. The warps of a block take different keys of
// one key head, or with many requests different key heads of the same keys (neighbours
// in the cache). 64 requests of 4100 keys, 4 key heads of 128: 107 us, 5.0 TB/s, set by
// the bytes in flight; 32-byte loads a lane were slower (174 us for 136 at the time).
// One request of 2052 keys: 14 us with its rows from DRAM, 9 us from L2.
//
// A request's keys are split over the blocks of a cluster (up to 16) when the
// requests alone do not fill the SMs; the partial maxima, sums and outputs meet
// through distributed shared memory and are added in rank order.
#include <cooperative_groups.h>

#include "scan_window_step.h"

namespace scan {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16* p, bool on) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (on) asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "l"(p));
  return v;
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// ROWS: 8 or 16 query heads a warp (the fragments' second eight rows are empty at 8).
// WH: key heads a block; the other warps share a head's keys.
template <int DP, int ROWS, int WH>
__global__ void __launch_bounds__(32 * kWarps, ROWS == 8 ? 3 : 2) window_step_kernel(const WinStepArgs a) {
  using bf16 = __nv_bfloat16;
  constexpr int KK = DP / 32, HALF = DP / 64, WK = kWarps / WH;
  __shared__ float s_m[kWarps][ROWS], s_l[kWarps][ROWS];
  __shared__ float s_o[kWarps][ROWS][DP];
  __shared__ float b_m[WH][ROWS], b_l[WH][ROWS];
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int g = lane / 4, c = lane % 4;
  const int split = blockIdx.x, splits = gridDim.x;
  const int G = a.Hq / a.Hk, tiles = (G + ROWS - 1) / ROWS;
  const int wh = warp % WH, wk = warp / WH;  // this warp's key head, and its share of the keys
  const int hk0 = blockIdx.y / tiles * WH, hk = hk0 + wh, r0 = (blockIdx.y % tiles) * ROWS;  // heads r0.. of the group
  const int rows = G - r0 < ROWS ? G - r0 : ROWS;
  const int64_t b = blockIdx.z;
  const int64_t slot = a.slots ? (int64_t)a.slots[b] : b, pos = a.pos[b];
  // output row r of key head x of the block
  const auto out = [&](int x, int r) {
    return static_cast<bf16*>(a.o.ptr) + b * a.o.stride_b + ((int64_t)(hk0 + x) * G + r0 + r) * a.o.stride_h;
  };
  if (slot < 0 || slot >= a.n_slots || pos < 0) {  // an idle request (the whole cluster)
    if (split == 0)
      for (int i = threadIdx.x; i < WH * rows * a.D; i += 32 * kWarps)
        out(i / a.D / rows, i / a.D % rows)[i % a.D] = __float2bfloat16_rn(0.f);
    return;
  }
  const int64_t at = pos < a.S ? pos : a.S + (pos - a.S) % a.W;
  const int64_t n = pos + 1 < a.cap ? pos + 1 : a.cap;
  const int64_t row = (int64_t)a.Hk * a.D;
  bf16* const kc = static_cast<bf16*>(a.kc) + slot * a.cap * row + (int64_t)hk * a.D;
  bf16* const vc = static_cast<bf16*>(a.vc) + slot * a.cap * row + (int64_t)hk * a.D;
  const bf16* const kn = static_cast<const bf16*>(a.k.ptr) + b * a.k.stride_b + hk * a.k.stride_h;
  const bf16* const vn = static_cast<const bf16*>(a.v.ptr) + b * a.v.stride_b + hk * a.v.stride_h;
  // the new token joins the cache; its row is read from k and v, never from there
  if (split == 0 && r0 == 0 && wk == 0)
    for (int i = lane; i < a.D; i += 32) kc[at * row + i] = kn[i], vc[at * row + i] = vn[i];

  // queries as the left operand: rows g and g + 8
  uint4 q[KK], q8[KK];
  {
    const bf16* qp = static_cast<const bf16*>(a.q.ptr) + b * a.q.stride_b + ((int64_t)hk * G + r0) * a.q.stride_h;
#pragma unroll
    for (int k = 0; k < KK; ++k) {
      const int d = 32 * k + 8 * c;
      q[k] = ld16(qp + g * a.q.stride_h + d, g < rows && d < a.D);
      q8[k] = ROWS == 16 ? ld16(qp + (g + 8) * a.q.stride_h + d, g + 8 < rows && d < a.D) : make_uint4(0, 0, 0, 0);
    }
  }
  const float sl2 = a.scale * 1.44269504088896341f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[HALF][8][4];
#pragma unroll
  for (int h = 0; h < HALF; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[h][j][x] = 0.f;

  const int64_t groups = (n + 15) / 16, per = (groups + splits - 1) / splits;
  const int64_t first = split * per, last = first + per < groups ? first + per : groups;
  uint4 kv[2][KK], vv[4][HALF];
  const auto load_k = [&](int64_t t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t j = t * 16 + 8 * x + g;
      const bf16* p = j == at ? kn : kc + j * row;
#pragma unroll
      for (int k = 0; k < KK; ++k) kv[x][k] = ld16(p + 32 * k + 8 * c, t < last && j < n && 32 * k + 8 * c < a.D);
    }
  };
  const auto load_v = [&](int64_t t) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t j = t * 16 + 2 * c + (x & 1) + 8 * (x >> 1);
      const bf16* p = j == at ? vn : vc + j * row;
#pragma unroll
      for (int h = 0; h < HALF; ++h) vv[x][h] = ld16(p + 64 * h + 8 * g, t < last && j < n && 64 * h + 8 * g < a.D);
    }
  };
  load_k(first + wk);
  load_v(first + wk);
#pragma unroll 1
  for (int64_t t = first + wk; t < last; t += WK) {
    const int64_t j0 = t * 16;
    float s[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
#pragma unroll
      for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        mma16816(s[x], q[k].x, q8[k].x, q[k].y, q8[k].y, kv[x][k].x, kv[x][k].y);
        mma16816(s[x], q[k].z, q8[k].z, q[k].w, q8[k].w, kv[x][k].z, kv[x][k].w);
      }
    }
    load_k(t + WK);  // on its way while the weights are taken and used
    // s[x][y], s[x][2 + y]: heads g and g + 8, key j0 + 8 x + 2 c + y
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (j0 + 8 * x + 2 * c + y >= n) s[x][y] = s[x][2 + y] = -INFINITY;
    float p[2][4];
#pragma unroll
    for (int h = 0; h < ROWS / 8; ++h) {
      float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m[h], top * sl2);
      const float from = mn == -INFINITY ? 0.f : mn, keep = ex2(m[h] - from);
      m[h] = mn;
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) sum += p[x][2 * h + y] = ex2(fmaf(s[x][2 * h + y], sl2, -from));
      l[h] = l[h] * keep + sum;
#pragma unroll
      for (int i = 0; i < HALF; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[i][j][2 * h] *= keep;
          acc[i][j][2 * h + 1] *= keep;
        }
    }
    // (weights as bf16, as the values they multiply: off by 2^-9 of themselves at most; l is
    // the sum of the unrounded ones)
    const uint32_t a0 = pack2(p[0][0], p[0][1]), a2 = pack2(p[1][0], p[1][1]);
    const uint32_t a1 = ROWS == 16 ? pack2(p[0][2], p[0][3]) : 0u, a3 = ROWS == 16 ? pack2(p[1][2], p[1][3]) : 0u;
#pragma unroll
    for (int i = 0; i < HALF; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
        mma16816(acc[i][j], a0, a1, a2, a3, __byte_perm(word(vv[0][i], j / 2), word(vv[1][i], j / 2), sel),
                 __byte_perm(word(vv[2][i], j / 2), word(vv[3][i], j / 2), sel));
      }
    load_v(t + WK);
  }
  // the warps' parts, then the block's
#pragma unroll
  for (int h = 0; h < ROWS / 8; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (c == 0) s_m[warp][8 * h + g] = m[h], s_l[warp][8 * h + g] = l[h];
#pragma unroll
    for (int i = 0; i < HALF; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s_o[warp][8 * h + g][64 * i + 16 * c + j] = acc[i][j][2 * h];
        s_o[warp][8 * h + g][64 * i + 16 * c + 8 + j] = acc[i][j][2 * h + 1];
      }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < WH * ROWS * DP; i += 32 * kWarps) {
    const int x = i / DP / ROWS, r = i / DP % ROWS, d = i % DP;
    float top = s_m[x][r];
#pragma unroll
    for (int w = 1; w < WK; ++w) top = fmaxf(top, s_m[x + w * WH][r]);
    const float from = top == -INFINITY ? 0.f : top;
    float sum = 0.f, e = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float f = ex2(s_m[x + w * WH][r] - from);
      sum = fmaf(s_l[x + w * WH][r], f, sum);
      e = fmaf(s_o[x + w * WH][r][d], f, e);
    }
    if (splits == 1) {
      if (r < rows && d < a.D) out(x, r)[d] = __float2bfloat16_rn(e / sum);
    } else {
      s_o[x][r][d] = e;  // read by no other thread
      if (d == 0) b_m[x][r] = top, b_l[x][r] = sum;
    }
  }
  if (splits == 1) return;
  // the cluster's parts: rank by rank, each block a share of the outputs
  cluster.sync();
  for (int i = split * 32 * kWarps + threadIdx.x; i < WH * rows * DP; i += splits * 32 * kWarps) {
    const int x = i / DP / rows, r = i / DP % rows, d = i % DP;
    float top = -INFINITY;
    for (int k = 0; k < splits; ++k) top = fmaxf(top, *cluster.map_shared_rank(&b_m[x][r], k));
    float sum = 0.f, e = 0.f;
    for (int k = 0; k < splits; ++k) {
      const float f = ex2(*cluster.map_shared_rank(&b_m[x][r], k) - top);
      sum = fmaf(*cluster.map_shared_rank(&b_l[x][r], k), f, sum);
      e = fmaf(*cluster.map_shared_rank(&s_o[x][r][d], k), f, e);
    }
    if (d < a.D) out(x, r)[d] = __float2bfloat16_rn(e / sum);
  }
  cluster.sync();  // no block leaves while its part may be read
}

template <int DP, int ROWS, int WH>
cudaError_t launch_step(const WinStepArgs& a, int64_t B, int splits, cudaStream_t s) {
  const int G = a.Hq / a.Hk, tiles = (G + ROWS - 1) / ROWS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(splits, (unsigned)(a.Hk / WH * tiles), (unsigned)B);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = splits;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (splits > 8) {
    const cudaError_t e = cudaFuncSetAttribute(window_step_kernel<DP, ROWS, WH>,
                                               cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, window_step_kernel<DP, ROWS, WH>, a);
}

// Rows of 16-byte pieces that this kernel's loads can address.
bool aligned16(const scan_view4& v) {
  return (uintptr_t)v.ptr % 16 == 0 && v.stride_b % 8 == 0 && v.stride_h % 8 == 0;
}

}  // namespace

bool window_step_fits(const WinStepArgs& a, scan_dtype dt) {
  return dt == SCAN_BF16 && aligned16(a.q) && aligned16(a.k) && aligned16(a.v);
}

namespace {

template <int DP, int ROWS>
cudaError_t launch_heads(const WinStepArgs& a, int64_t B, int wh, int splits, cudaStream_t s) {
  if (wh == 4) return launch_step<DP, ROWS, 4>(a, B, splits, s);
  if (wh == 2) return launch_step<DP, ROWS, 2>(a, B, splits, s);
  return launch_step<DP, ROWS, 1>(a, B, splits, s);
}

}  // namespace

// A block takes one key head, its four warps a quarter of the keys each, where these
// blocks are resident at once, and else up to four key heads, a warp each. In us by key
// heads a block (4 / 1), 4 key heads of 128: 1 request of 2052 keys 21 / 11, 8 of them
// 25 / 17, 32 of 4100 keys 63 / 55, 64 of them 110 / 106, 100 of them 182 / 139; past
// what is resident, 128 of them 199 / 237.
// Splits of a request's keys: as many as stay resident at once (two to three blocks
// an SM, on 128 of the SMs: clusters do not fill every group of SMs), as long as a
// warp has two steps of 16 keys. 64 requests of 4100 keys and 4 key heads a block, in us
// by splits: 332 (1), 184, 141, 114, 120, 111 (6), 138 (7: a second round of clusters).
cudaError_t launch_window_step(const WinStepArgs& a, int64_t B, cudaStream_t s) {
  const int G = a.Hq / a.Hk, rows = G <= 8 ? 8 : 16, tiles = (G + rows - 1) / rows, per_sm = rows == 8 ? 3 : 2;
  const int wh = B * a.Hk * tiles <= per_sm * 152 ? 1 : a.Hk % 4 == 0 ? 4 : a.Hk % 2 == 0 ? 2 : 1;
  const int64_t blocks = B * (a.Hk / wh) * tiles, slots = per_sm * 128;
  int64_t n = slots / blocks;
  const int64_t most = a.cap / (2 * 16 * (kWarps / wh));
  n = n > most ? most : n;
  const int splits = (int)(n < 1 ? 1 : n > 16 ? 16 : n);
  if (a.D <= 64)
    return rows == 8 ? launch_heads<64, 8>(a, B, wh, splits, s) : launch_heads<64, 16>(a, B, wh, splits, s);
  return rows == 8 ? launch_heads<128, 8>(a, B, wh, splits, s) : launch_heads<128, 16>(a, B, wh, splits, s);
}

}  // namespace scan
