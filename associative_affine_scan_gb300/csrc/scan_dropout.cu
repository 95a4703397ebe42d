// scan_dropout.cu -- dropout whose mask is never stored: y = x / (1 - p) where the
// generator keeps an element, else 0. The backward is the same pass over the
// gradient: it draws the same numbers from the same seed and call.
//
// One read and one write of each element, bound by DRAM; the generator's ten rounds
// serve eight elements (some twelve instructions an element with the conversion,
// about half of what the SMs can issue in the time that bf16 elements take to move).
// 8 x 4096 x 2048 bf16: 45.6 us, 5.9 TB/s.
#include "scan_mixer.h"
#include "scan_philox.cuh"

namespace scan {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // blocks of eight elements a thread, all their loads on the way at once

struct DropArgs {
  const void* x;
  void* y;
  int64_t x_sb, x_st, y_sb, y_st;
  int64_t T, C, n;  // n = B T C elements
  Drop drop;
};

template <typename T>
struct Eight;  // eight elements in memory
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ static void store(float* p, const float2 (&v)[4]) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(v[2].x, v[2].y, v[3].x, v[3].y));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float2 (&v)[4]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
  }
};

// ROWS: rows of C elements (a multiple of 8) at any 16-byte strides; else n elements
// one after the other. The last, shorter block of those goes element by element.
template <typename T, bool ROWS>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropArgs a) {
  uint64_t seed, call;
  a.drop.read(&seed, &call);
  const int64_t first = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x, whole = a.n / 8;
  const T* const x = static_cast<const T*>(a.x);
  T* const y = static_cast<T*>(a.y);
  Eight<T> e[kUnroll];
  int64_t to[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t blk = first + i * kThreads;
    int64_t from = to[i] = blk * 8;
    if (ROWS) {
      const int64_t row = blk / (a.C / 8), c = (blk - row * (a.C / 8)) * 8, b = row / a.T, t = row - b * a.T;
      from = b * a.x_sb + t * a.x_st + c;
      to[i] = b * a.y_sb + t * a.y_st + c;
    }
    if (blk < whole) e[i].load(x + from);
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int64_t blk = first + i * kThreads;
    if (blk < whole) {
      float2 v[4];
      e[i].get(v);
      if (a.drop.limit) drop8(v, a.drop, (uint64_t)blk, call, seed);
      Eight<T>::store(y + to[i], v);
    } else if (!ROWS && blk == whole && a.n % 8) {
      const int left = (int)(a.n % 8);
      float2 v[4];
#pragma unroll
      for (int j = 0; j < 8; ++j) (j % 2 ? v[j / 2].y : v[j / 2].x) = j < left ? to_f32(x[blk * 8 + j]) : 0.f;
      if (a.drop.limit) drop8(v, a.drop, (uint64_t)blk, call, seed);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) y[blk * 8 + j] = from_f32<T>(j % 2 ? v[j / 2].y : v[j / 2].x);
    }
  }
}

// Any strides and alignment: a thread has a block's eight elements one by one.
template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_general(const DropArgs a) {
  uint64_t seed, call;
  a.drop.read(&seed, &call);
  const int64_t blk = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (blk * 8 >= a.n) return;
  int64_t row = blk * 8 / a.C, c = blk * 8 - row * a.C, b = row / a.T, t = row - b * a.T;
  const int left = a.n - blk * 8 < 8 ? (int)(a.n - blk * 8) : 8;
  float2 v[4];
  int64_t to[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float& e = j % 2 ? v[j / 2].y : v[j / 2].x;
    e = 0.f;
    to[j] = b * a.y_sb + t * a.y_st + c;
    if (j < left) e = to_f32(static_cast<const T*>(a.x)[b * a.x_sb + t * a.x_st + c]);
    if (++c == a.C) {
      c = 0;
      if (++t == a.T) t = 0, ++b;
    }
  }
  if (a.drop.limit) drop8(v, a.drop, (uint64_t)blk, call, seed);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < left) static_cast<T*>(a.y)[to[j]] = from_f32<T>(j % 2 ? v[j / 2].y : v[j / 2].x);
}

bool on16(const void* p) { return (uintptr_t)p % 16 == 0; }

template <typename T>
cudaError_t launch(DropArgs a, int64_t B, cudaStream_t s) {
  constexpr int64_t E = 16 / sizeof(T);
  const auto flat = [&](int64_t sb, int64_t st) {
    return (a.T == 1 || st == a.C) && (B == 1 || sb == a.T * a.C);
  };
  const bool aligned = on16(a.x) && on16(a.y);
  const int64_t per = kThreads * kUnroll, blocks = (a.n / 8 + (a.n % 8 ? 1 : 0) + per - 1) / per;
  if (aligned && flat(a.x_sb, a.x_st) && flat(a.y_sb, a.y_st)) {
    dropout_kernel<T, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  } else if (aligned && a.C % 8 == 0 && a.x_sb % E == 0 && a.x_st % E == 0 && a.y_sb % E == 0 && a.y_st % E == 0) {
    dropout_kernel<T, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  } else {
    dropout_general<T><<<(unsigned)((a.n + 8 * kThreads - 1) / (8 * kThreads)), kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

scan_status dropout(const scan_view4* x, const scan_view4* y, int64_t B, int64_t T, int64_t C, double p,
                    uint64_t seed, uint64_t call, const int64_t* rng, scan_dtype dt, cudaStream_t s) {
  if (dt != SCAN_F32 && dt != SCAN_BF16) return SCAN_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || C < 0 || !(p >= 0. && p <= 1.)) return SCAN_ERR_INVALID_ARG;
  if (B == 0 || T == 0 || C == 0) return SCAN_OK;
  if (!x || !x->ptr || !y || !y->ptr) return SCAN_ERR_INVALID_ARG;
  if ((uintptr_t)rng % 8) return SCAN_ERR_ALIGNMENT;
  // a grid's blocks, of eight elements a thread at least
  if ((double)B * (double)T * (double)C > (double)(1LL << 41)) return SCAN_ERR_UNSUPPORTED;
  // an axis of one element has no stride of its own
  const auto sb = [&](const scan_view4* v) { return B > 1 ? v->stride_b : 0; };
  const auto st = [&](const scan_view4* v) { return T > 1 ? v->stride_t : 0; };
  DropArgs a{x->ptr, y->ptr, sb(x), st(x), sb(y), st(y), T, C, B * T * C, make_drop(p, seed, call, rng)};
  const cudaError_t e = dt == SCAN_BF16 ? launch<__nv_bfloat16>(a, B, s) : launch<float>(a, B, s);
  return e == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // namespace
}  // namespace scan

using namespace scan;

extern "C" {

scan_status dropout_fwd(const scan_view4* x, const scan_view4* y, int64_t B, int64_t T, int64_t C, double p,
                        uint64_t seed, uint64_t call, const int64_t* rng, scan_dtype dt, cudaStream_t stream) {
  return dropout(x, y, B, T, C, p, seed, call, rng, dt, stream);
}

scan_status dropout_bwd(const scan_view4* dy, const scan_view4* dx, int64_t B, int64_t T, int64_t C, double p,
                        uint64_t seed, uint64_t call, const int64_t* rng, scan_dtype dt, cudaStream_t stream) {
  return dropout(dy, dx, B, T, C, p, seed, call, rng, dt, stream);
}

}  // extern "C"
