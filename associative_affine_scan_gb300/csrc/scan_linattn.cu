// scan_linattn.cu -- linear attention with a decay for each head: the entry
// points, the general path and the form for single tokens.
//
//   S_t = lambda S_{t-1} + k_t v_t^T  (Dk x Dv),   o_t = scale q_t S_t
//
// General path (fp32 operands, operands that tensor copies cannot address, and
// short rows): the recurrence itself. Columns of S are independent, so a block
// owns one (sequence, head) and 32 columns, four threads a column with a quarter
// of its rows each in registers; 16 steps of the operands are staged in shared
// memory at a time. It is bound by the latency of a step (about 5 operations per
// state element in four threads), not by memory: 0.6 us a step for 16 heads of
// 128 x 128 in bf16, 0.9 us in fp32; 5.8 us for 1024.
// lambda is rounded once, and a state multiplied by it t times would be off by t times
// that: what the rounding leaves out, delta = lambda / fl(lambda) - 1, is taken out of
// what enters the state at step t, as (1 + delta)^-t, and put back where the state is
// read, so that only the roundings of the steps remain (memories of 20 to 260 steps: states
// and outputs are 1.3e-5 off without and 4e-7 with; 1 to 6 % of the time).
//
// Step: the state is read and written once, so it is bound by DRAM (8 Dk Dv
// bytes a head against 5 Dk Dv operations): 1024 heads of 128 x 128 in 19 us, 7.0 TB/s
// (the last writes are still in L2 when it ends). A block takes one (request, head);
// thread x owns four columns, thread y every 8th or 16th row, so all loads and
// stores are whole 512-byte rows, and the read-out's sum over rows ends in shared
// memory. lambda is held in two parts, so that the states of many tokens do not gather
// its rounding (1e-5 over a memory of 260 tokens).
#include "scan_linattn_tc.h"
#include "scan_mixer.h"

namespace scan {
namespace {

// log(lambda / lam) of a lambda that was rounded to lam: lam - 1 is exact where it is used.
// A state that loses most of itself every step gathers no such error.
__device__ __forceinline__ float rounding_of(float lam, float log_decay) {
  return lam > 0.25f && lam < 4.f ? log_decay - log1pf(lam - 1.f) : 0.f;
}

constexpr int kCols = 32;   // columns of S a block of the general path owns
constexpr int kSteps = 16;  // steps staged in shared memory
constexpr int kSettle = 1 << 20;  // after so many steps the powers of 1 + delta start anew

template <typename T, int KP>
__global__ void __launch_bounds__(4 * kCols, KP == 64 ? 8 : 6) linattn_general_kernel(const LinArgs a) {
  const LinPass& p = a.pass[blockIdx.z];
  const int v0 = blockIdx.y * kCols;
  if (v0 >= p.V) return;
  __shared__ float s1[kSteps][KP], s2[kSteps][KP], s3[kSteps][kCols];
  __shared__ float drift, taken[kSteps], back[kSteps];  // powers of lambda / fl(lambda), see above
  const int h = (int)(blockIdx.x % a.H);
  const int64_t sb = blockIdx.x / a.H;  // batch row, or packed sequence
  int64_t beg = 0, end = a.T;
  if (a.cu) {
    seq_bounds(a.cu, (int)sb, a.T, &beg, &end);
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) check_seqlens(a.cu, a.n_seqs, a.T, a.hdr);
  }
  const int64_t b = a.cu ? 0 : sb;
  const View<const T> x1{static_cast<const T*>(p.x1.ptr), p.x1.stride_b, p.x1.stride_t, p.x1.stride_h};
  const View<const T> x2{static_cast<const T*>(p.x2.ptr), p.x2.stride_b, p.x2.stride_t, p.x2.stride_h};
  const View<const T> x3{static_cast<const T*>(p.x3.ptr), p.x3.stride_b, p.x3.stride_t, p.x3.stride_h};
  const View<T> out{static_cast<T*>(p.out.ptr), p.out.stride_b, p.out.stride_t, p.out.stride_h};
  const float lam = expf(a.log_decay[h]);
  if (threadIdx.x == 0) drift = rounding_of(lam, a.log_decay[h]);  // in shared memory for the few who use it
  const int skip = p.reverse ? 0 : 1;  // multiplications that step 0's entry is ahead of the initial state
  const int col = threadIdx.x >> 2, part = threadIdx.x & 3, c = v0 + col;
  // rows 16 i + 4 part + r of S, r < 4
  float S[KP / 4];
  const int64_t st = (sb * a.H + h) * (int64_t)p.K * p.V;
#pragma unroll
  for (int i = 0; i < KP / 4; ++i) {
    const int k = 16 * (i / 4) + 4 * part + i % 4;
    S[i] = 0.f;
    if (p.s_in && k < p.K && c < p.V)
      S[i] = p.s_in_mul * p.s_in[st + (p.s_in_t ? (int64_t)c * p.K + k : (int64_t)k * p.V + c)];
  }
  const int64_t n = end - beg;
  int64_t from = 0;  // the steps before are settled: the powers stay near 1
  for (int64_t t0 = 0; t0 < n; t0 += kSteps) {
    if (t0 - from == kSettle) {
      const float all = expf(drift * (float)kSettle);
#pragma unroll
      for (int i = 0; i < KP / 4; ++i) S[i] *= all;
      from = t0;
    }
    const int m = (int)(n - t0 < kSteps ? n - t0 : kSteps);
    __syncthreads();
    for (int i = threadIdx.x; i < kSteps * KP; i += 4 * kCols) {
      const int t = i / KP, k = i % KP;
      float u = 0.f, w = 0.f;
      if (t < m && k < p.K) {
        const int64_t at = p.reverse ? end - 1 - (t0 + t) : beg + t0 + t;
        u = to_f32(x1.row(b, at, h)[k]);
        w = to_f32(x2.row(b, at, h)[k]);
      }
      s1[t][k] = u;
      s2[t][k] = w;
    }
    for (int i = threadIdx.x; i < kSteps * kCols; i += 4 * kCols) {
      const int t = i / kCols, k = i % kCols;
      const int64_t at = p.reverse ? end - 1 - (t0 + t) : beg + t0 + t;
      s3[t][k] = t < m && v0 + k < p.V ? to_f32(x3.row(b, at, h)[v0 + k]) : 0.f;
    }
    if (threadIdx.x < 2 * kSteps) {
      const float f = drift * (float)(t0 - from + threadIdx.x % kSteps + skip);
      if (threadIdx.x < kSteps) taken[threadIdx.x] = expf(-f);
      else back[threadIdx.x - kSteps] = a.scale * expf(f);
    }
    __syncthreads();
    for (int t = 0; t < m; ++t) {
      const float v = s3[t][col] * taken[t];
      float o = 0.f;
#pragma unroll
      for (int i = 0; i < KP / 16; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(&s1[t][16 * i + 4 * part]);
        const float4 k = *reinterpret_cast<const float4*>(&s2[t][16 * i + 4 * part]);
        const float qa[4] = {q.x, q.y, q.z, q.w}, ka[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float& e = S[4 * i + r];
          if (!p.reverse) e *= lam;
          e = fmaf(ka[r], v, e);
          o = fmaf(qa[r], e, o);
          if (p.reverse) e *= lam;
        }
      }
      o += __shfl_xor_sync(0xffffffffu, o, 1);
      o += __shfl_xor_sync(0xffffffffu, o, 2);
      if (part == 0 && c < p.V) {
        const int64_t at = p.reverse ? end - 1 - (t0 + t) : beg + t0 + t;
        out.row(b, at, h)[c] = from_f32<T>(o * back[t]);
      }
    }
  }
  if (p.s_out) {
    const float mul = n > 0 ? p.s_out_mul * expf(drift * (float)(n - from)) : p.s_out_mul;
#pragma unroll
    for (int i = 0; i < KP / 4; ++i) {
      const int k = 16 * (i / 4) + 4 * part + i % 4;
      if (k < p.K && c < p.V) p.s_out[st + (int64_t)k * p.V + c] = mul * S[i];
    }
  }
}

template <typename T>
cudaError_t launch_general_t(const LinArgs& a, cudaStream_t s) {
  int K = 0, V = 0;
  for (int i = 0; i < a.npass; ++i) {
    K = a.pass[i].K > K ? a.pass[i].K : K;
    V = a.pass[i].V > V ? a.pass[i].V : V;
  }
  const int64_t n = (a.cu ? a.n_seqs : a.B) * a.H;
  const dim3 grid((unsigned)n, (V + kCols - 1) / kCols, a.npass);
  if (K <= 64) linattn_general_kernel<T, 64><<<grid, 4 * kCols, 0, s>>>(a);
  else linattn_general_kernel<T, 128><<<grid, 4 * kCols, 0, s>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------

struct StepArgs {
  scan_view4 q, k, v, o;
  const float* log_decay;
  float* state;
  const int32_t* slots;
  int64_t n_slots;
  int H, Dk, Dv;
  float scale;
};

// Columns 4 x.. of the state in thread x (Dv / 4 threads a row, at most 32), row y,
// y + rows, ... in thread row y.
template <typename T>
__global__ void __launch_bounds__(256) linattn_step_kernel(const StepArgs a) {
  const int h = (int)(blockIdx.x % a.H);
  const int64_t b = blockIdx.x / a.H;
  const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
  const int cx = threadIdx.x % 32, ry = threadIdx.x / 32;  // eight rows at a time
  const int c = 4 * cx;
  T* o = static_cast<T*>(a.o.ptr) + b * a.o.stride_b + h * a.o.stride_h;
  if (slot < 0 || slot >= a.n_slots) {  // no state: the request is idle
    if (threadIdx.x < a.Dv) o[threadIdx.x] = from_f32<T>(0.f);
    return;
  }
  __shared__ float sq[kMixMaxDim], sk[kMixMaxDim];
  __shared__ float4 red[8][32];
  const T* q = static_cast<const T*>(a.q.ptr) + b * a.q.stride_b + h * a.q.stride_h;
  const T* k = static_cast<const T*>(a.k.ptr) + b * a.k.stride_b + h * a.k.stride_h;
  const T* v = static_cast<const T*>(a.v.ptr) + b * a.v.stride_b + h * a.v.stride_h;
  float* S = a.state + ((slot * a.H + h) * a.Dk) * (int64_t)a.Dv;
  const bool on = c < a.Dv;
  // the whole state is in flight before anything is used: 16 rows a thread at most
  float4 e[kMixMaxDim / 8];
#pragma unroll
  for (int i = 0; i < kMixMaxDim / 8; ++i) {
    const int r = ry + 8 * i;
    if (on && r < a.Dk) e[i] = __ldcs(reinterpret_cast<const float4*>(S + (int64_t)r * a.Dv + c));
  }
  for (int i = threadIdx.x; i < a.Dk; i += 256) {
    sq[i] = to_f32(q[i]);
    sk[i] = to_f32(k[i]);
  }
  const float lam = expf(a.log_decay[h]), low = lam * rounding_of(lam, a.log_decay[h]);  // lambda in two parts
  float4 vv = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) vv = make_float4(to_f32(v[c]), to_f32(v[c + 1]), to_f32(v[c + 2]), to_f32(v[c + 3]));
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kMixMaxDim / 8; ++i) {
    const int r = ry + 8 * i;
    if (on && r < a.Dk) {
      const float kk = sk[r], qq = sq[r];
      float4 x = e[i];
      x.x = fmaf(kk, vv.x, fmaf(x.x, lam, x.x * low));
      x.y = fmaf(kk, vv.y, fmaf(x.y, lam, x.y * low));
      x.z = fmaf(kk, vv.z, fmaf(x.z, lam, x.z * low));
      x.w = fmaf(kk, vv.w, fmaf(x.w, lam, x.w * low));
      __stcs(reinterpret_cast<float4*>(S + (int64_t)r * a.Dv + c), x);
      acc.x = fmaf(qq, x.x, acc.x);
      acc.y = fmaf(qq, x.y, acc.y);
      acc.z = fmaf(qq, x.z, acc.z);
      acc.w = fmaf(qq, x.w, acc.w);
    }
  }
  red[ry][cx] = acc;
  __syncthreads();
  if (threadIdx.x < a.Dv) {
    float s = 0.f;
    for (int y = 0; y < 8; ++y) s += reinterpret_cast<const float*>(&red[y][0])[threadIdx.x];
    o[threadIdx.x] = from_f32<T>(s * a.scale);
  }
}

scan_status lin_common(const LinArgs& a, scan_dtype dt, int64_t H, int64_t Dk, int64_t Dv) {
  if (dt != SCAN_F32 && dt != SCAN_BF16) return SCAN_ERR_INVALID_ARG;
  if (a.B < 0 || a.T < 0 || H < 0 || Dk < 1 || Dv < 1 || a.n_seqs < 0) return SCAN_ERR_INVALID_ARG;
  if (a.cu && (a.B != 1 || (a.n_seqs == 0 && a.T > 0))) return SCAN_ERR_INVALID_ARG;
  if (!(a.scale > 0.f) || !(a.scale < INFINITY)) return SCAN_ERR_INVALID_ARG;
  if (Dk > kMixMaxDim || Dv > kMixMaxDim || Dk % 8 || Dv % 8) return SCAN_ERR_UNSUPPORTED;
  const int64_t n = a.cu ? a.n_seqs : a.B;
  if (n > 0x7fffffffLL || H > 0x7fffffffLL || n * H > 0x7fffffffLL || a.T > (1LL << 40))
    return SCAN_ERR_UNSUPPORTED;
  if (a.cu && a.T > 0x7fffffffLL) return SCAN_ERR_UNSUPPORTED;
  return SCAN_OK;
}

bool given(const scan_view4* v) { return v && v->ptr; }

cudaError_t lin_launch(const LinArgs& a, scan_dtype dt, cudaStream_t s) {
  if (linattn_tc_fits(a, dt)) return launch_linattn_tc(a, s);
  return launch_linattn_general(a, dt, s);
}

scan_status lin_workspace(LinArgs* a, void* ws, size_t bytes, size_t need) {
  if (!ws || (uintptr_t)ws % 16 || bytes < need) return SCAN_ERR_WORKSPACE;
  a->hdr = static_cast<WsHeader*>(ws);
  a->ws = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeaderBytes);
  return SCAN_OK;
}

}  // namespace

cudaError_t launch_linattn_general(const LinArgs& a, scan_dtype dt, cudaStream_t s) {
  return dt == SCAN_BF16 ? launch_general_t<__nv_bfloat16>(a, s) : launch_general_t<float>(a, s);
}

}  // namespace scan

using namespace scan;

extern "C" {

size_t linattn_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                               int64_t n_seqs) {
  if (B < 0 || T < 0 || H < 0 || n_seqs < 0 || Dk < 1 || Dv < 1 || Dk > kMixMaxDim || Dv > kMixMaxDim)
    return 0;
  return kWsHeaderBytes + linattn_tc_workspace_bytes(B, T, H, Dk, Dv, n_seqs);
}

scan_status linattn_fwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                        const float* log_decay, const float* h0, const int32_t* cu_seqlens,
                        int32_t n_seqs, const scan_view4* o, float* hT, int64_t B, int64_t T,
                        int64_t H, int64_t Dk, int64_t Dv, float scale, scan_dtype dt,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  LinArgs a{};
  a.cu = cu_seqlens;
  a.n_seqs = n_seqs;
  a.B = B;
  a.T = T;
  a.H = (int)H;
  a.scale = scale;
  a.log_decay = log_decay;
  scan_status st = lin_common(a, dt, H, Dk, Dv);
  if (st != SCAN_OK) return st;
  const int64_t n = cu_seqlens ? n_seqs : B;
  if (n * H == 0) return SCAN_OK;
  if (!log_decay) return SCAN_ERR_INVALID_ARG;
  if (T > 0 && (!given(q) || !given(k) || !given(v) || !given(o))) return SCAN_ERR_INVALID_ARG;
  st = lin_workspace(&a, workspace, workspace_bytes,
                     linattn_workspace_bytes(B, T, H, Dk, Dv, cu_seqlens ? n_seqs : 0));
  if (st != SCAN_OK) return st;
  LinPass& p = a.pass[0];
  if (T > 0) {
    p.x1 = *q;
    p.x2 = *k;
    p.x3 = *v;
    p.out = *o;
  }
  p.s_in = h0;
  p.s_in_mul = 1.f;
  p.s_out = hT;
  p.s_out_mul = 1.f;
  p.K = (int)Dk;
  p.V = (int)Dv;
  a.npass = 1;
  return lin_launch(a, dt, stream) == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status linattn_bwd(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                        const float* log_decay, const float* h0, const int32_t* cu_seqlens,
                        int32_t n_seqs, const scan_view4* dout, const float* dhT,
                        const scan_view4* dq, const scan_view4* dk, const scan_view4* dv, float* dh0,
                        int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv, float scale,
                        scan_dtype dt, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
  LinArgs a{};
  a.cu = cu_seqlens;
  a.n_seqs = n_seqs;
  a.B = B;
  a.T = T;
  a.H = (int)H;
  a.scale = scale;
  a.log_decay = log_decay;
  scan_status st = lin_common(a, dt, H, Dk, Dv);
  if (st != SCAN_OK) return st;
  const int64_t n = cu_seqlens ? n_seqs : B;
  if (n * H == 0) return SCAN_OK;
  if (!log_decay) return SCAN_ERR_INVALID_ARG;
  if (T > 0 && (!given(q) || !given(k) || !given(v) || !given(dout) || !given(dq) || !given(dk) ||
                !given(dv)))
    return SCAN_ERR_INVALID_ARG;
  st = lin_workspace(&a, workspace, workspace_bytes,
                     linattn_workspace_bytes(B, T, H, Dk, Dv, cu_seqlens ? n_seqs : 0));
  if (st != SCAN_OK) return st;
  // Every pass's sums leave the kernel times `scale`; a state that comes in from
  // outside without that factor is divided by it first.
  const float inv = 1.f / scale;
  LinPass &pq = a.pass[0], &pk = a.pass[1], &pv = a.pass[2];
  if (T > 0) {
    pq.x1 = *dout;
    pq.x2 = *v;
    pq.x3 = *k;
    pq.out = *dq;
    pk.x1 = *v;
    pk.x2 = *dout;
    pk.x3 = *q;
    pk.out = *dk;
    pv.x1 = *k;
    pv.x2 = *q;
    pv.x3 = *dout;
    pv.out = *dv;
  }
  pq.s_in = h0;
  pq.s_in_t = 1;
  pq.s_in_mul = 1.f;
  pk.s_in = pv.s_in = dhT;
  pk.s_in_t = 1;
  pk.s_in_mul = pv.s_in_mul = inv;
  pv.s_out = dh0;
  pv.s_out_mul = scale;
  pq.K = pk.K = (int)Dv;
  pq.V = pk.V = (int)Dk;
  pv.K = (int)Dk;
  pv.V = (int)Dv;
  pk.reverse = pv.reverse = 1;
  a.npass = 3;
  return lin_launch(a, dt, stream) == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

scan_status linattn_step(const scan_view4* q, const scan_view4* k, const scan_view4* v,
                         const float* log_decay, float* state, const int32_t* slots, int64_t n_slots,
                         const scan_view4* o, int64_t B, int64_t H, int64_t Dk, int64_t Dv,
                         float scale, scan_dtype dt, cudaStream_t stream) {
  LinArgs c{};
  c.B = B;
  c.scale = scale;
  const scan_status st = lin_common(c, dt, H, Dk, Dv);
  if (st != SCAN_OK) return st;
  if (n_slots < 0) return SCAN_ERR_INVALID_ARG;
  if (B * H == 0) return SCAN_OK;
  if (!given(q) || !given(k) || !given(v) || !given(o) || !log_decay || !state)
    return SCAN_ERR_INVALID_ARG;
  if (!slots && n_slots < B) return SCAN_ERR_INVALID_ARG;
  if ((uintptr_t)state % 16) return SCAN_ERR_ALIGNMENT;
  StepArgs a{*q, *k, *v, *o, log_decay, state, slots, n_slots, (int)H, (int)Dk, (int)Dv, scale};
  if (dt == SCAN_BF16)
    linattn_step_kernel<__nv_bfloat16><<<(unsigned)(B * H), 256, 0, stream>>>(a);
  else
    linattn_step_kernel<float><<<(unsigned)(B * H), 256, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? SCAN_OK : SCAN_ERR_CUDA;
}

}  // extern "C"
