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
// address. Products are of fp32 accuracy on the tensor cores: each factor is the sum of
// two tf32 numbers, hi of its upper 11 bits and lo of what is left, and a b = hi hi + hi lo
// + lo hi (what is left out is 2^-22 of a b, as the rounding of lo is), summed in fp32.
// Three m16n8k8 products are 169 multiply-adds a cycle and SM, where fp32 arithmetic
// has 128 and reads more of its factors from shared memory. A warp has 16 rows; tiles lie
// in shared memory row by row, with a pitch that puts the elements of a fragment into
// different banks both as rows (q k) and as columns (p v): the summed index of the
// second product runs over the keys in the order in which the first one's results lie
// with the threads.
// fp32, 2 x 777 queries, 1031 keys, 12 heads of 64 over 4: 134 us, 37 TFLOP/s of fp32
// products (fp32 arithmetic would take 66 us at its peak). Bound by instruction issue and its
// waits: each warp splits the tile's factors for itself, and products are a ninth of its
// instructions (44 % of what the tensor cores do in this form).
#include "scan_cross.h"
#include "scan_cross_tc.h"

namespace scan {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kOwn = 16 * kWarps;  // rows that a block owns
constexpr int kOther = 32;         // rows of the other sequence that it takes at a time

template <int DP>
constexpr int kPitch = DP + 4;

template <typename T>
__device__ __forceinline__ View<T> vw(const scan_view4& v) {
  return View<T>{static_cast<T*>(v.ptr), v.stride_b, v.stride_t, v.stride_h};
}

// Rows [t0, t0 + ROWS) of one head as fp32, zeros from row `end` and column D on. fp32
// rows come by asynchronous copies, of 16 bytes where they lie on 16 bytes.
template <typename T, int DP, int ROWS>
__device__ __forceinline__ void load_rows(float* dst, const View<const T>& v, int64_t b, int64_t t0, int64_t end,
                                          int64_t h, int D, bool on16) {
  if constexpr (sizeof(T) == 4) {
    const int step = on16 ? 4 : 1, per = DP / step;
    for (int i = threadIdx.x; i < ROWS * per; i += kThreads) {
      const int r = i / per, c = i % per * step;
      const bool on = t0 + r < end && c < D;
      const T* const p = v.row(b, on ? t0 + r : 0, h) + (on ? c : 0);
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst + r * kPitch<DP> + c);
      if (!on) {  // (nothing is read: the operand may be empty)
        if (step == 4) *reinterpret_cast<float4*>(dst + r * kPitch<DP> + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        else dst[r * kPitch<DP> + c] = 0.f;
      } else if (step == 4) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
      } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(p) : "memory");
      }
    }
  } else {
    for (int i = threadIdx.x; i < ROWS * DP; i += kThreads) {
      const int r = i / DP, c = i % DP;
      dst[r * kPitch<DP> + c] = t0 + r < end && c < D ? to_f32(v.row(b, t0 + r, h)[c]) : 0.f;
    }
  }
}
__device__ __forceinline__ void loads_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void loads_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
bool rows_on_16(const scan_view4& v, int64_t B, int64_t T, int64_t H) {
  return (uintptr_t)v.ptr % 16 == 0 && (B <= 1 || v.stride_b % 4 == 0) && (T <= 1 || v.stride_t % 4 == 0) &&
         (H <= 1 || v.stride_h % 4 == 0);
}

// x = hi + lo, hi rounded to the 11 bits of a tf32 number (the products ignore what lo has
// beyond its own).
__device__ __forceinline__ void split(float x, uint32_t* hi, uint32_t* lo) {
  *hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  *lo = __float_as_uint(x - __uint_as_float(*hi));
}
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A thread of a warp has rows g and g + 8 and columns 2 c, 2 c + 1 of each 16 x 8 result.
struct Lane {
  int g, c;
  __device__ Lane() : g(threadIdx.x % 32 / 4), c(threadIdx.x % 4) {}
};

// The products add to their sums by cutting off, not by rounding, which a long sum would
// show (7.6e-6 of an output over 1031 keys). So sums run over one tile only, the small
// terms by themselves, and are added to the others by rounding additions.

// acc[j] += rows of `a` (16, from the warp's first) times rows 8 j .. of `b`, over D columns.
template <int DP>
__device__ __forceinline__ void rows_by_rows(float (&acc)[kOther / 8][4], const float* a, const float* b, int D) {
  constexpr int N = kOther / 8;
  const Lane w;
  float small[N][4] = {};
#pragma unroll 2
  for (int k = 0; k < D; k += 8) {
    uint32_t hi[4], lo[4], bh[N][2], bl[N][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) split(a[(w.g + 8 * (i & 1)) * kPitch<DP> + k + w.c + 4 * (i >> 1)], &hi[i], &lo[i]);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i) split(b[(8 * j + w.g) * kPitch<DP> + k + w.c + 4 * i], &bh[j][i], &bl[j][i]);
#pragma unroll
    for (int j = 0; j < N; ++j) mma1688(small[j], lo, bh[j]);
#pragma unroll
    for (int j = 0; j < N; ++j) mma1688(acc[j], hi, bh[j]);
#pragma unroll
    for (int j = 0; j < N; ++j) mma1688(small[j], hi, bl[j]);
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] += small[j][i];
}
// acc[i] += p times columns 8 i .. of `b`, over its rows; p as rows_by_rows left it.
template <int DP>
__device__ __forceinline__ void weights_by_columns(float (&acc)[DP / 8][4], const float (&p)[kOther / 8][4], const float* b,
                                                   int D) {
  constexpr int N = kOther / 8;
  const Lane w;
  uint32_t hi[N][4], lo[N][4];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    split(p[j][0], &hi[j][0], &lo[j][0]);
    split(p[j][2], &hi[j][1], &lo[j][1]);
    split(p[j][1], &hi[j][2], &lo[j][2]);
    split(p[j][3], &hi[j][3], &lo[j][3]);
  }
#pragma unroll
  for (int i0 = 0; i0 < DP / 8; i0 += 4) {  // 32 columns at a time
    if (8 * i0 >= D) break;
    float sum[4][4] = {}, small[4][4] = {};
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const float* const at = b + (8 * j + 2 * w.c) * kPitch<DP> + 8 * i0 + w.g;
      uint32_t bh[4][2], bl[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int y = 0; y < 2; ++y) split(at[8 * i + y * kPitch<DP>], &bh[i][y], &bl[i][y]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mma1688(small[i], lo[j], bh[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mma1688(sum[i], hi[j], bh[i]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mma1688(small[i], hi[j], bl[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int y = 0; y < 4; ++y) acc[i0 + i][y] += sum[i][y] + small[i][y];
  }
}
// The warp's 16 rows from row t0 on, rows g times f[0] and g + 8 times f[1].
template <typename T, int DP>
__device__ __forceinline__ void write_rows(const View<T>& out, const float (&acc)[DP / 8][4], int64_t b, int64_t t0,
                                           int64_t end, int64_t h, int D, const float (&f)[2]) {
  const Lane w;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int64_t t = t0 + w.g + 8 * y;
    if (t >= end) continue;
    T* const row = out.row(b, t, h) + 2 * w.c;
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
      if (8 * i < D) {
        row[8 * i] = from_f32<T>(acc[i][2 * y] * f[y]);
        row[8 * i + 1] = from_f32<T>(acc[i][2 * y + 1] * f[y]);
      }
  }
}
// Over the four threads of a row.
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Pairs of tiles (of two operands) that a walk holds at a time: the next one is on its way
// while this one is used, where shared memory has room for both and two blocks an SM.
template <int DP, int OWN>
constexpr int kStages = (OWN * kOwn + 4 * kOther) * kPitch<DP> * 4 <= (112 << 10) ? 2 : 1;
template <int DP, int OWN>
constexpr int kSmem = (OWN * kOwn + 2 * kStages<DP, OWN> * kOther) * kPitch<DP> * 4;

// Brings pair after pair of tiles to shared memory: use(x, y, n) with tile n of both.
template <int DP, int OWN, typename L, typename U>
__device__ __forceinline__ void walk(float* tiles, int64_t n, const L& load, const U& use) {
  constexpr int NS = kStages<DP, OWN>, size = kOther * kPitch<DP>;
  if (NS == 2 && n > 0) load(tiles, tiles + size, 0);
  loads_commit();
  for (int64_t i = 0; i < n; ++i) {
    float* const x = tiles + (NS == 2 ? (i & 1) * 2 * size : 0);
    if (NS == 1) {
      __syncthreads();  // the last tiles have been used
      load(x, x + size, i);
      loads_commit();
      loads_wait<0>();
    } else {
      float* const y = tiles + ((i + 1) & 1) * 2 * size;
      if (i > 0) __syncthreads();
      if (i + 1 < n) load(y, y + size, i + 1);
      loads_commit();
      loads_wait<1>();
    }
    __syncthreads();
    use(x, x + size, i);
  }
  loads_wait<0>();
}

// What a piece of a query tile's walk over the keys leaves of a row: the maximum and the sum
// of its weights, and the sum of its values, in the workspace.
struct Pieces {
  float *m, *l;     // [pieces][B][Hq][Tq]
  View<float> o;    // the first piece's [B, Tq, Hq, D]
  int64_t rows, size;  // rows and floats of o from piece to piece
};
__host__ __device__ inline Pieces pieces_at(const CrossArgs& a, int pieces) {
  const int64_t rows = a.B * a.Hq * a.Tq, stats = (rows * pieces + 3) / 4 * 4;
  return Pieces{a.ws, a.ws + stats, View<float>{a.ws + 2 * stats, a.Hq * a.Tq * a.D, a.D, a.Tq * a.D}, rows, rows * a.D};
}
size_t pieces_floats(int64_t B, int64_t Tq, int64_t Hq, int64_t D, int pieces) {
  return pieces > 1 ? (size_t)pieces * (size_t)(B * Hq * Tq) * (size_t)(D + 2) + 8 : 0;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) cross_fwd_general(const CrossArgs a, int on16, int pieces) {
  extern __shared__ float4 raw[];
  asm volatile("griddepcontrol.launch_dependents;");
  float *const sq = reinterpret_cast<float*>(raw), *const tiles = sq + kOwn * kPitch<DP>;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  CrossRows g;
  const int h = blockIdx.y % a.Hq, hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.y / a.Hq;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kOwn, false, &g)) return;
  const Lane w;
  const int warp = threadIdx.x / 32;
  const View<const T> k = vw<const T>(a.k), v = vw<const T>(a.v);
  load_rows<T, DP, kOwn>(sq, vw<const T>(a.q), b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D, on16);
  const float* const own = sq + 16 * warp * kPitch<DP>;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[DP / 8][4] = {};
  const int64_t all = (g.nk + kOther - 1) / kOther, first = all * blockIdx.z / pieces, last = all * (blockIdx.z + 1) / pieces;
  walk<DP, 1>(
      tiles, last - first,
      [&](float* x, float* y, int64_t i) {
        const int64_t t = g.kbeg + (first + i) * kOther;
        load_rows<T, DP, kOther>(x, k, b, t, g.kbeg + g.nk, hk, a.D, on16);
        load_rows<T, DP, kOther>(y, v, b, t, g.kbeg + g.nk, hk, a.D, on16);
      },
      [&](const float* sk, const float* sv, int64_t i) {
        float s[kOther / 8][4] = {};
        rows_by_rows<DP>(s, own, sk, a.D);
        const int64_t left = g.nk - (first + i) * kOther;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < kOther / 8; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float& e = s[j][2 * y + z];
              e = 8 * j + 2 * w.c + z < left ? e * a.scale : -INFINITY;
              top = fmaxf(top, e);
            }
          const float mn = fmaxf(m[y], row_max(top)), base = mn == -INFINITY ? 0.f : mn;
          const float keep = expf(m[y] - base);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < kOther / 8; ++j)
#pragma unroll
            for (int z = 0; z < 2; ++z) sum += s[j][2 * y + z] = expf(s[j][2 * y + z] - base);
          l[y] = l[y] * keep + sum;
          m[y] = mn;
#pragma unroll
          for (int x = 0; x < DP / 8; ++x) o[x][2 * y] *= keep, o[x][2 * y + 1] *= keep;
        }
        weights_by_columns<DP>(o, s, sv, a.D);
      });
  float f[2] = {1.f, 1.f};
  if (pieces > 1) {
    Pieces p = pieces_at(a, pieces);
    p.o.p += blockIdx.z * p.size;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] = row_sum(l[y]);
      const int64_t t = g.t0 + 16 * warp + w.g + 8 * y, at = blockIdx.z * p.rows + (b * a.Hq + h) * a.Tq + g.qbeg + t;
      if (w.c == 0 && t < g.nq) p.m[at] = m[y], p.l[at] = l[y];
    }
    write_rows<float, DP>(p.o, o, b, g.qbeg + g.t0 + 16 * warp, g.qbeg + g.nq, h, a.D, f);
    return;
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    l[y] = row_sum(l[y]);
    f[y] = l[y] == 0.f ? 0.f : 1.f / l[y];  // l is 0 where there is no key; NaN stays
    const int64_t t = g.t0 + 16 * warp + w.g + 8 * y;
    if (w.c == 0 && t < g.nq)
      a.lse[(b * a.Hq + h) * a.Tq + g.qbeg + t] = l[y] == 0.f ? -INFINITY : m[y] + logf(l[y]);
  }
  write_rows<T, DP>(vw<T>(a.o), o, b, g.qbeg + g.t0 + 16 * warp, g.qbeg + g.nq, h, a.D, f);
}

// The pieces of a row, added in order: a warp a row, four columns a lane; eight blocks a
// tile of 64 rows (with one, 24 us of a call of 142).
template <typename T>
__global__ void __launch_bounds__(256) cross_join_general(const CrossArgs a, int pieces) {
  CrossRows g;
  const int h = blockIdx.y % a.Hq, lane = threadIdx.x % 32;
  const int64_t b = blockIdx.y / a.Hq;
  const bool any = cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kOwn, false, &g);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!any) return;
  const Pieces p = pieces_at(a, pieces);
  const int64_t t = g.t0 + 8 * blockIdx.z + threadIdx.x / 32, at = (b * a.Hq + h) * a.Tq + g.qbeg + t;
  if (t >= g.nq) return;
  float top = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int z = 0; z < pieces; ++z) top = fmaxf(top, p.m[z * p.rows + at]);
  const float base = top == -INFINITY ? 0.f : top;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int z = 0; z < pieces; ++z) {
    float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
    if (4 * lane < a.D) e = *reinterpret_cast<const float4*>(p.o.row(b, g.qbeg + t, h) + z * p.size + 4 * lane);
    const float f = expf(p.m[z * p.rows + at] - base);
    sum = fmaf(p.l[z * p.rows + at], f, sum);
    o.x = fmaf(e.x, f, o.x), o.y = fmaf(e.y, f, o.y), o.z = fmaf(e.z, f, o.z), o.w = fmaf(e.w, f, o.w);
  }
  const float r = sum == 0.f ? 0.f : 1.f / sum;  // no key; NaN stays
  if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : top + logf(sum);
  if (4 * lane < a.D) {
    T* const row = vw<T>(a.o).row(b, g.qbeg + t, h) + 4 * lane;
    row[0] = from_f32<T>(o.x * r), row[1] = from_f32<T>(o.y * r), row[2] = from_f32<T>(o.z * r), row[3] = from_f32<T>(o.w * r);
  }
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

// A tile of queries against the keys, or a piece of them (blockIdx.z).
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) cross_dq_general(const CrossArgs a, int on16, int pieces) {
  extern __shared__ float4 raw[];
  asm volatile("griddepcontrol.launch_dependents;");
  float *const sq = reinterpret_cast<float*>(raw), *const sd = sq + kOwn * kPitch<DP>, *const tiles = sd + kOwn * kPitch<DP>;
  CrossRows g;
  const int h = blockIdx.y % a.Hq, hk = h / (a.Hq / a.Hk);
  const int64_t b = blockIdx.y / a.Hq;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kOwn, false, &g)) return;
  const Lane w;
  const int warp = threadIdx.x / 32;
  const View<const T> k = vw<const T>(a.k), v = vw<const T>(a.v);
  load_rows<T, DP, kOwn>(sq, vw<const T>(a.q), b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D, on16);
  load_rows<T, DP, kOwn>(sd, vw<const T>(a.dout), b, g.qbeg + g.t0, g.qbeg + g.nq, h, a.D, on16);
  float lse[2], delta[2], dq[DP / 8][4] = {};
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int64_t t = g.t0 + 16 * warp + w.g + 8 * y, at = (b * a.Hq + h) * a.Tq + g.qbeg + t;
    lse[y] = t < g.nq ? a.lse[at] : INFINITY;
    delta[y] = t < g.nq ? a.delta[at] : 0.f;
  }
  const int64_t all = (g.nk + kOther - 1) / kOther, first = all * blockIdx.z / pieces, last = all * (blockIdx.z + 1) / pieces;
  walk<DP, 2>(
      tiles, last - first,
      [&](float* x, float* y, int64_t i) {
        const int64_t t = g.kbeg + (first + i) * kOther;
        load_rows<T, DP, kOther>(x, k, b, t, g.kbeg + g.nk, hk, a.D, on16);
        load_rows<T, DP, kOther>(y, v, b, t, g.kbeg + g.nk, hk, a.D, on16);
      },
      [&](const float* sk, const float* sv, int64_t i) {
        float s[kOther / 8][4] = {}, dp[kOther / 8][4] = {};
        rows_by_rows<DP>(s, sq + 16 * warp * kPitch<DP>, sk, a.D);
        rows_by_rows<DP>(dp, sd + 16 * warp * kPitch<DP>, sv, a.D);
        const int64_t left = g.nk - (first + i) * kOther;
#pragma unroll
        for (int j = 0; j < kOther / 8; ++j)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            s[j][z] = 8 * j + 2 * w.c + z % 2 < left
                          ? expf(s[j][z] * a.scale - lse[z / 2]) * (dp[j][z] - delta[z / 2])
                          : 0.f;
        weights_by_columns<DP>(dq, s, sk, a.D);
      });
  const float f[2] = {a.scale, a.scale};
  const int64_t t0 = g.qbeg + g.t0 + 16 * warp;
  if (pieces > 1) {
    const View<float> part{a.ws + blockIdx.z * (a.B * a.Hq * a.Tq * a.D), a.Hq * a.Tq * a.D, a.D, a.Tq * a.D};
    write_rows<float, DP>(part, dq, b, t0, g.qbeg + g.nq, h, a.D, f);
  } else {
    write_rows<T, DP>(vw<T>(a.dq), dq, b, t0, g.qbeg + g.nq, h, a.D, f);
  }
}

// The pieces of dq, added in order: a warp a row, four columns a lane; eight blocks a tile.
template <typename T>
__global__ void __launch_bounds__(256) cross_dq_join_general(const CrossArgs a, int pieces) {
  CrossRows g;
  const int h = blockIdx.y % a.Hq, c = threadIdx.x % 32 * 4;
  const int64_t b = blockIdx.y / a.Hq;
  const bool any = cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x, kOwn, false, &g);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = g.t0 + 8 * blockIdx.z + threadIdx.x / 32;
  if (!any || t >= g.nq || c >= a.D) return;
  const float* const from = a.ws + ((b * a.Hq + h) * a.Tq + g.qbeg + t) * a.D + c;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int z = 0; z < pieces; ++z) {
    const float4 e = *reinterpret_cast<const float4*>(from + z * (a.B * a.Hq * a.Tq * a.D));
    s.x += e.x, s.y += e.y, s.z += e.z, s.w += e.w;
  }
  T* const row = vw<T>(a.dq).row(b, g.qbeg + t, h) + c;
  row[0] = from_f32<T>(s.x), row[1] = from_f32<T>(s.y), row[2] = from_f32<T>(s.z), row[3] = from_f32<T>(s.w);
}

// A tile of keys against every query, over the heads that share it, or one of `pieces`
// parts of that walk, whose sums go to the workspace. Rows past a sequence's keys
// (padding) get zeros.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) cross_dkv_general(const CrossArgs a, int on16, int pieces) {
  extern __shared__ float4 raw[];
  float *const sk = reinterpret_cast<float*>(raw), *const sv = sk + kOwn * kPitch<DP>, *const tiles = sv + kOwn * kPitch<DP>;
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32)
    check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  CrossRows g;
  const int hk = blockIdx.y % a.Hk, G = a.Hq / a.Hk, piece = blockIdx.x % pieces;
  const int64_t b = blockIdx.y / a.Hk;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, b, blockIdx.x / pieces, kOwn, true, &g)) return;
  const Lane w;
  const int warp = threadIdx.x / 32;
  const View<const T> q = vw<const T>(a.q), dout = vw<const T>(a.dout);
  load_rows<T, DP, kOwn>(sk, vw<const T>(a.k), b, g.kbeg + g.t0, g.kbeg + g.nk, hk, a.D, on16);
  load_rows<T, DP, kOwn>(sv, vw<const T>(a.v), b, g.kbeg + g.t0, g.kbeg + g.nk, hk, a.D, on16);
  float dk[DP / 8][4] = {}, dv[DP / 8][4] = {};
  const int64_t per = g.t0 < g.nk ? (g.nq + kOther - 1) / kOther : 0;
  const int64_t first = per * G * piece / pieces, last = per * G * (piece + 1) / pieces;
  walk<DP, 2>(
      tiles, last - first,
      [&](float* x, float* y, int64_t i) {
        const int64_t h = hk * G + (first + i) / per, t0 = (first + i) % per * kOther;
        load_rows<T, DP, kOther>(x, q, b, g.qbeg + t0, g.qbeg + g.nq, h, a.D, on16);
        load_rows<T, DP, kOther>(y, dout, b, g.qbeg + t0, g.qbeg + g.nq, h, a.D, on16);
      },
      [&](const float* sq, const float* sd, int64_t i) {
        const int64_t h = hk * G + (first + i) / per, t0 = (first + i) % per * kOther;
        float s[kOther / 8][4] = {}, dp[kOther / 8][4] = {};
        rows_by_rows<DP>(s, sk + 16 * warp * kPitch<DP>, sq, a.D);
        rows_by_rows<DP>(dp, sv + 16 * warp * kPitch<DP>, sd, a.D);
#pragma unroll
        for (int j = 0; j < kOther / 8; ++j)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int64_t t = t0 + 8 * j + 2 * w.c + z, at = (b * a.Hq + h) * a.Tq + g.qbeg + t;
            const bool on = t < g.nq;
            const float lse = on ? a.lse[at] : INFINITY, delta = on ? a.delta[at] : 0.f;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float &e = s[j][2 * y + z], &f = dp[j][2 * y + z];
              e = on && g.t0 + 16 * warp + w.g + 8 * y < g.nk ? expf(e * a.scale - lse) : 0.f;
              f = e * (f - delta);
            }
          }
        weights_by_columns<DP>(dv, s, sd, a.D);
        weights_by_columns<DP>(dk, dp, sq, a.D);
      });
  const int64_t rows = a.cu_q ? g.nk : a.Tk, t0 = g.kbeg + g.t0 + 16 * warp;
  const float one[2] = {1.f, 1.f}, f[2] = {a.scale, a.scale};
  if (pieces > 1) {
    const int64_t row = (int64_t)a.Hk * a.D, all = a.B * a.Tk * row;
    const View<float> pk{a.ws + 2 * piece * all, a.Tk * row, row, a.D}, pv{pk.p + all, a.Tk * row, row, a.D};
    write_rows<float, DP>(pk, dk, b, t0, g.kbeg + rows, hk, a.D, f);
    write_rows<float, DP>(pv, dv, b, t0, g.kbeg + rows, hk, a.D, one);
  } else {
    write_rows<T, DP>(vw<T>(a.dk), dk, b, t0, g.kbeg + rows, hk, a.D, f);
    write_rows<T, DP>(vw<T>(a.dv), dv, b, t0, g.kbeg + rows, hk, a.D, one);
  }
}

// The pieces' sums, added in order: an element of dk and of dv a thread.
template <typename T>
__global__ void __launch_bounds__(256) cross_pieces_general(const CrossArgs a, int pieces) {
  const int64_t all = a.B * a.Tk * a.Hk * a.D, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= all) return;
  float k = 0.f, v = 0.f;
#pragma unroll 4
  for (int p = 0; p < pieces; ++p) {
    k += a.ws[2 * p * all + i];
    v += a.ws[(2 * p + 1) * all + i];
  }
  const int64_t d = i % a.D, h = i / a.D % a.Hk, t = i / a.D / a.Hk % a.Tk, b = i / a.D / a.Hk / a.Tk;
  vw<T>(a.dk).row(b, t, h)[d] = from_f32<T>(k);
  vw<T>(a.dv).row(b, t, h)[d] = from_f32<T>(v);
}

// Pieces of a key tile's walk: as many as fill the SMs four times over, of four tiles of
// queries at least.
int general_pieces(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t n_seqs) {
  if (Hk < 1 || B < 1 || Tk < 1) return 1;
  const int64_t blocks = ((Tk + kOwn - 1) / kOwn + n_seqs) * B * Hk;
  const int64_t walk = Hq / Hk * ((Tq + kOther - 1) / kOther) / (n_seqs > 1 ? n_seqs : 1);
  int64_t p = 4 * 152 / blocks;
  p = p < walk / 4 ? p : walk / 4;
  return (int)(p < 1 ? 1 : p);
}

// Pieces of a query tile's walk: as many as give every SM eight blocks, of 128 keys at least
// (2 x 777 rows of 12 heads over 1031 keys, 312 tiles, in us: 162 whole or up to four blocks
// an SM, of which some SMs get one more than most; 151 with six, 134 with eight, 132 with
// twelve). Of dq as well (900 queries of five packed sequences over 3000 keys, 8 heads of
// 96, forward and backward: 584 us with dq whole, 387 so).
int fwd_pieces(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t n_seqs) {
  if (Hq < 1 || B < 1 || Tq < 1) return 1;
  const int64_t blocks = ((Tq + kOwn - 1) / kOwn + n_seqs) * B * Hq;
  const int64_t walk = Tk / (n_seqs > 1 ? n_seqs : 1);
  int64_t p = 8 * 152 / blocks;
  p = p < walk / 128 ? p : walk / 128;
  return (int)(p < 1 ? 1 : p);
}

template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int DP>
cudaError_t general_fwd(const CrossArgs& a, cudaStream_t s) {
  constexpr int smem = kSmem<DP, 1>;
  cudaError_t e = allow_smem(cross_fwd_general<T, DP>, smem);
  if (e != cudaSuccess) return e;
  const int on16 = rows_on_16(a.q, a.B, a.Tq, a.Hq) && rows_on_16(a.k, a.B, a.Tk, a.Hk) && rows_on_16(a.v, a.B, a.Tk, a.Hk);
  const int64_t tiles = (a.Tq + kOwn - 1) / kOwn + (a.cu_q ? a.n_seqs : 0);
  const int pieces = fwd_pieces(a.B, a.Tq, a.Tk, a.Hq, a.n_seqs);
  const dim3 grid((unsigned)tiles, (unsigned)(a.B * a.Hq), (unsigned)pieces);
  cross_fwd_general<T, DP><<<grid, kThreads, smem, s>>>(a, on16, pieces);
  e = cudaGetLastError();
  if (e != cudaSuccess || pieces == 1) return e;
  return launch_early(cross_join_general<T>, dim3(grid.x, grid.y, kOwn / 8), 256, 0, s, a, pieces);
}

template <typename T, int DP>
cudaError_t general_bwd(const CrossArgs& a, cudaStream_t s) {
  constexpr int smem = kSmem<DP, 2>;
  cudaError_t e = allow_smem(cross_dq_general<T, DP>, smem);
  if (e == cudaSuccess) e = allow_smem(cross_dkv_general<T, DP>, smem);
  if (e != cudaSuccess) return e;
  const int on16 = rows_on_16(a.q, a.B, a.Tq, a.Hq) && rows_on_16(a.dout, a.B, a.Tq, a.Hq) &&
                   rows_on_16(a.k, a.B, a.Tk, a.Hk) && rows_on_16(a.v, a.B, a.Tk, a.Hk);
  const int64_t rows = a.B * a.Tq * a.Hq, extra = a.cu_q ? a.n_seqs : 0;
  const int64_t tq = (a.Tq + kOwn - 1) / kOwn + extra, tk = (a.Tk + kOwn - 1) / kOwn + extra;
  if (rows > 0) {
    cross_delta_general<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a, rows);
    const int parts = fwd_pieces(a.B, a.Tq, a.Tk, a.Hq, a.n_seqs);
    const dim3 grid((unsigned)tq, (unsigned)(a.B * a.Hq), (unsigned)parts);
    cross_dq_general<T, DP><<<grid, kThreads, smem, s>>>(a, on16, parts);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (parts > 1) {
      e = launch_early(cross_dq_join_general<T>, dim3(grid.x, grid.y, kOwn / 8), 256, 0, s, a, parts);
      if (e != cudaSuccess) return e;
    }
  }
  if (a.Tk < 1 || a.Hk < 1) return cudaGetLastError();
  const int pieces = general_pieces(a.B, a.Tq, a.Tk, a.Hq, a.Hk, a.n_seqs);
  cross_dkv_general<T, DP><<<dim3((unsigned)(tk * pieces), (unsigned)(a.B * a.Hk)), kThreads, smem, s>>>(a, on16, pieces);
  if (pieces > 1)
    cross_pieces_general<T><<<(unsigned)((a.B * a.Tk * a.Hk * a.D + 255) / 256), 256, 0, s>>>(a, pieces);
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
  if (Tq > 0x7fffffffLL || Tk > 0x7fffffffLL) return SCAN_ERR_UNSUPPORTED;
  const int64_t H = Hq > Hk ? Hq : Hk;  // (no query heads may read some key heads)
  if (B > 0x7fffffffLL || H > 0x7fffffffLL || B * H > 0x7fffffffLL) return SCAN_ERR_UNSUPPORTED;  // a grid's blocks
  return SCAN_OK;
}

scan_status cross_common(CrossArgs* a, const int32_t* lens, const int32_t* cu_q, const int32_t* cu_k, int32_t n_seqs,
                         int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, float scale,
                         scan_dtype dt) {
  const scan_status st = cross_sizes(B, Tq, Tk, Hq, Hk, D, scale, dt);
  if (st != SCAN_OK) return st;
  if (B * Hq > 65535 || B * Hk > 65535) return SCAN_ERR_UNSUPPORTED;  // a grid's second axis
  if (B * Hq * Tq > (1LL << 33)) return SCAN_ERR_UNSUPPORTED;  // blocks of the row sums
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
  if (!backward) return kWsHeaderBytes + pieces_floats(B, Tq, Hq, D, fwd_pieces(B, Tq, Tk, Hq, n_seqs)) * 4;
  const size_t tc = cross_tc_bwd_floats(B, Tq, Tk, Hq, D, n_seqs);
  const int pieces = general_pieces(B, Tq, Tk, Hq, Hk, n_seqs);
  const int parts = fwd_pieces(B, Tq, Tk, Hq, n_seqs);  // of dq, in the same place before
  const size_t of_dq = parts > 1 ? (size_t)parts * (size_t)(B * Hq * Tq * D) : 0;
  size_t general = pieces > 1 ? (size_t)pieces * 2 * (size_t)(B * Tk * Hk * D) : 0;
  if (of_dq > general) general = of_dq;
  return kWsHeaderBytes + round_up((size_t)(B * Hq * Tq) * 4, 256) + (tc > general ? tc : general) * 4;
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
  a.ws = a.delta;
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
  if (B * (Hq * Tq + Hk * Tk) == 0) return SCAN_OK;
  if (Hq * Tq > 0 && (!given(q) || !given(o) || !given(dout) || !given(dq) || !lse)) return SCAN_ERR_INVALID_ARG;
  if (Hk * Tk > 0 && (!given(k) || !given(v) || !given(dk) || !given(dv))) return SCAN_ERR_INVALID_ARG;
  st = cross_workspace(&a, workspace, workspace_bytes, cross_attn_workspace_bytes(B, Tq, Tk, Hq, Hk, D, a.n_seqs, 1));
  if (st != SCAN_OK) return st;
  if (Hq * Tq > 0) a.q = *q, a.o = *o, a.dout = *dout, a.dq = *dq;
  if (Hk * Tk > 0) a.k = *k, a.v = *v, a.dk = *dk, a.dv = *dv;
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
