// scan_window_bwd.cu -- backward of sliding-window attention with first tokens
// that stay visible, on the tensor cores (bf16 operands).
//
//   p = 2^(scale log2(e) q k - lse log2(e)), ds = p (do v - delta), delta = do o
//   dv = sum p do, dk = scale sum ds q (over queries and the heads that share the
//   key head), dq = scale sum ds k (over keys)
//
// Two kernels, each with its sums in tensor memory and no sum across blocks: the
// five products become seven, but no result depends on the order in which blocks
// run and nothing is added in global memory. 2 x 4096 tokens, 16 query heads of 128
// over 4 key heads, window 1024: keys 157 us (0.77 PFLOP/s of seen pairs' four products),
// queries 132 us (0.69, three products), row sums 14 us, pieces 5 us.
//   keys:    a block owns 128 keys and walks the tiles of 128 queries that see
//            them: S = k q^T, dP = v do^T, dv += P do, dk += dS q. Keys are the
//            rows of S, so P and dS (bf16, over S and dP in tensor memory) are
//            read as they lie by the two second products.
//   queries: a block owns 128 queries of a head and walks the key tiles they see:
//            S = q k^T, dP = do v^T, dq += dS k. It runs first: where the queries see one
//            tile, it forms their delta anew from p and dP, for the keys' kernel as well.
// The order of issue keeps the tensor cores busy while two warpgroups turn S and
// dP into P and dS, half of the columns each: the first product of the next tile
// is issued between the two that wait for them. Both are bound by that chain: the tensor
// cores (512 cycles a product at D = 128) are busy for 51 % (keys) and 39 % (queries) of
// a block's cycles; 280 blocks of keys on 152 SMs leave a quarter of the time idle besides,
// which smaller pieces would fill at the price of sums in memory. The queries' kernel issues dP from a
// warp of its own (141 -> 132 us on 2 x 4096 x 16 heads, window 1024); the same
// in the keys' kernel, whose two chains then alternate, took 170 us for 160.
//
// The tile of keys that holds the first tokens is seen by every later query: its
// walk is cut into pieces of about the length of any other tile's, whose partial
// sums (fp32, workspace) are added in order by a last kernel.
#include "scan_tc.cuh"
#include "scan_window_phases.h"
#include "scan_window_tc.h"

namespace scan {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kThreads = 10 * 32;    // two warpgroups of softmax, copies, products
constexpr int kThreadsDq = 11 * 32;  // and a second product warp
constexpr uint32_t kHalf = kRows * kPitch;

struct BwdArgs {
  CUtensorMap q, k, v, dout, dq, dk, dv;
  __nv_bfloat16 *dqp, *dkp, *dvp;
  int64_t dq_sb, dq_st, dq_sh, dk_sb, dk_st, dk_sh, dv_sb, dv_st, dv_sh;
  const float* lse;
  float* delta;
  float* part;  // [B, Hk, pieces, sink tiles, 2, 128, D]
  const int32_t* cu;
  WsHeader* hdr;
  int64_t Tq, Tk, W, S;
  int n_seqs, Hq, Hk, G, D;
  int sink_tiles, pieces;  // key tiles whose walk is cut (dense only), and into how many
  float sl2, scale;
};

template <int DP>
struct Plan {
  static constexpr int kTileBytes = kRows * DP * 2;
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kMisc = 4096;  // barriers, row statistics
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024 + (DP == 128 ? 2048 : kMisc);
};

// Rows [from, 128) of a tile to zeros, by 256 threads.
template <int DP>
__device__ __forceinline__ void clear_rows(uint32_t tile, int from, int t) {
  const int left = kRows - from;
  for (int i = t; i < left * 8 * (DP / 64); i += 256)
    st_shared16(tile + (i / 8 / left) * kHalf + (from + i / 8 % left) * kPitch + (i % 8) * 16, 0, 0, 0, 0);
  fence_async();
  __syncwarp();
}

// What a pair of bf16 numbers leaves of the numbers they were rounded from, as bf16.
__device__ __forceinline__ uint32_t rest_bf16(uint32_t h, float a, float b) {
  return pack_bf16(a - __uint_as_float(h << 16), b - __uint_as_float(h & 0xffff0000u));
}

// A row of D fp32 sums in tensor memory times f, as bf16: to a tile in shared
// memory, or straight to `out`.
template <int DP>
__device__ __forceinline__ void write_row(uint32_t tsum, float f, uint32_t tile, int r, bool direct, bool live,
                                          __nv_bfloat16* out, int D) {
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) {
    uint32_t o[32];
    tmem_ld32(tsum + 32 * i, o);
    ld_wait();
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
      uint32_t w[4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        w[y] = pack_bf16(__uint_as_float(o[c + 2 * y]) * f, __uint_as_float(o[c + 2 * y + 1]) * f);
      const int col = 32 * i + c;
      if (direct) {
        if (live && col < D) *reinterpret_cast<uint4*>(out + col) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        st_shared16(swizzled(tile + (col / 64) * kHalf, r, col % 64 / 8), w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// ---------------------------------------------------------------------------

struct DeltaArgs {
  const __nv_bfloat16 *o, *d;
  int64_t o_sb, o_st, o_sh, d_sb, d_st, d_sh;
  float* delta;
  int64_t T, rows;
  int H, D;
};

// delta = sum of dout o of every row: 16 lanes of 16 bytes a row, four rows in
// flight a lane. Bound by DRAM: 67 MB in 14.5 us, 4.6 TB/s.
__global__ void __launch_bounds__(256) window_delta16_kernel(const DeltaArgs a) {
  const int lane = threadIdx.x % 16;
  const int64_t r0 = ((int64_t)blockIdx.x * 16 + threadIdx.x / 16) * 4;
  int64_t tok = r0 / a.H, b = tok / a.T, t = tok - b * a.T;
  int h = (int)(r0 - tok * a.H);
  int64_t at[4];
  uint4 x[4], y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    at[i] = (b * a.H + h) * a.T + t;
    if (r0 + i < a.rows && 8 * lane < a.D) {
      x[i] = *reinterpret_cast<const uint4*>(a.o + b * a.o_sb + t * a.o_st + h * a.o_sh + 8 * lane);
      y[i] = *reinterpret_cast<const uint4*>(a.d + b * a.d_sb + t * a.d_st + h * a.d_sh + 8 * lane);
    }
    if (++h == a.H) {
      h = 0;
      if (++t == a.T) t = 0, ++b;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, v[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s = fmaf(__uint_as_float(u[k] << 16), __uint_as_float(v[k] << 16), s);
      s = fmaf(__uint_as_float(u[k] & 0xffff0000u), __uint_as_float(v[k] & 0xffff0000u), s);
    }
#pragma unroll
    for (int k = 8; k; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    if (lane == 0 && r0 + i < a.rows) a.delta[at[i]] = s;
  }
}

template <int DP, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) window_dkv_kernel(const __grid_constant__ BwdArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t sK = base, sV = base + P::kTileBytes, sR = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bKV = bars, bFull = bars + 8, bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS, bDp = bS + 8,
                 bP = bDp + 8, bDs = bP + 8, bEnd = bDs + 8, bOut = bEnd + 8, bLse = bOut + 16,
                 bDelta = bLse + 8;
  uint32_t* const tmem_ptr = misc + 64;
  uint32_t* const stop_flag = misc + 65;
  float* const s_lse = reinterpret_cast<float*>(misc + 72);  // lse log2(e) of a tile's queries
  float* const s_delta = s_lse + kRows;

  if (a.cu && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) check_seqlens(a.cu, a.n_seqs, a.Tk, a.hdr);
  // which keys: the cut tiles' pieces first, then the others
  const int hk = blockIdx.y % a.Hk, b = blockIdx.y / a.Hk;
  int piece = -1;
  int64_t tile = blockIdx.x;
  if (a.pieces > 1) {
    const int cut = a.sink_tiles * a.pieces;
    if (blockIdx.x < cut) {
      piece = blockIdx.x % a.pieces;
      tile = blockIdx.x / a.pieces;
    } else {
      tile = blockIdx.x - cut + a.sink_tiles;
    }
  }
  TileRows g;
  if (!tile_rows(a.cu, a.n_seqs, a.Tq, a.Tk, tile, kRows, &g)) return;
  // query tiles [lo, hi] that see a key of the tile, over the heads that share it
  const int64_t kend = g.t0 + kRows < g.nk ? g.t0 + kRows : g.nk;
  int64_t qa = g.t0 - g.off, qz = kend - 1 + a.W - 1 - g.off;
  qa = qa < 0 ? 0 : qa;
  if (g.t0 < a.S || qz > g.nq - 1) qz = g.nq - 1;
  const int64_t lo = qa / kRows;
  const int per = qz < qa ? 0 : (int)(qz / kRows - lo + 1);
  int u0 = 0, u1 = per * a.G;
  if (piece >= 0) {
    const int64_t total = u1;
    u0 = (int)(total * piece / a.pieces);
    u1 = (int)(total * (piece + 1) / a.pieces);
  }
  const int n = u1 - u0;
  const auto head = [&](int u) { return hk * a.G + (u0 + u) / per; };
  const auto qrow = [&](int u) { return (lo + (u0 + u) % per) * kRows; };

  // queries (u even) or output gradients of tile u / 2 into their slot
  const auto load = [&](int u) {
    const int sl = u % NS, t = (int)(g.qbeg + qrow(u / 2)), hq = head(u / 2);
    bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
    for (int i = 0; i < DP / 64; ++i)
      copy_in_4d(sR + sl * P::kTileBytes + i * kHalf, u & 1 ? &a.dout : &a.q, bFull + 8 * sl, 64 * i, hq, t, b);
  };
  // the copy warp sets the barriers up and starts the first copies while the others prepare
  if (warp == 8 && lane == 0) {
    *stop_flag = 0;
    bar_init(bKV, 1);
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 1);
    }
    bar_init(bS, 1);
    bar_init(bDp, 1);
    bar_init(bP, 8);
    bar_init(bDs, 8);
    bar_init(bEnd, 1);
    bar_init(bOut, 4);
    bar_init(bOut + 8, 4);
    bar_init(bLse, 4);
    bar_init(bDelta, 4);
    bar_init_fence();
    if (n > 0) {
      bar_expect(bKV, 2 * P::kTileBytes);
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        copy_in_4d(sK + i * kHalf, &a.k, bKV, 64 * i, hk, (int)(g.kbeg + g.t0), b);
        copy_in_4d(sV + i * kHalf, &a.v, bKV, 64 * i, hk, (int)(g.kbeg + g.t0), b);
      }
      for (int u = 0; u < NS && u < 2 * n; ++u) load(u);
    }
  }
  __syncwarp();
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *tmem_ptr, tS = tm, tDp = tm + 128, tDv = tm + 256, tDk = tm + 384;
  const Stop stop{stop_flag, a.hdr};

  if (warp == 8) {
    // ---- copies: keys and values once, then queries and output gradients
    if (lane == 0) {
      for (int u = NS; u < 2 * n; ++u) {
        if (!bar_wait(bEmpty + 8 * (u % NS), (u / NS - 1) & 1, stop)) break;
        load(u);
      }
    }
  } else if (warp == 9) {
    // ---- products
    if (n > 0) {
      const bool lead = lane == 0;
      constexpr uint32_t dS = product_desc(128, 128, false, false);
      constexpr uint32_t dO = product_desc(128, DP, false, true);
      const auto slot = [&](int u) { return kmajor(sR) + (u % NS) * (P::kTileBytes >> 4); };
      const auto slot_mn = [&](int u) { return mnmajor(sR, kHalf) + (u % NS) * (P::kTileBytes >> 4); };
      const auto full = [&](int u) { return warp_wait(bFull + 8 * (u % NS), (u / NS) & 1, stop); };
      // two halves of 64 query columns, each packed where its scores were
      const auto second = [&](uint32_t d, uint32_t w, uint32_t t, bool add) {
        mma_tn<64>(lead, d, w, t, dO, add);
        mma_tn<64>(lead, d, w + 64, t + (64 * kPitch >> 4), dO, true);
      };
      bool ok = warp_wait(bKV, 0, stop) && full(0) && full(1);
      if (ok) {
        mma_kk<DP, kHalf, kHalf>(lead, tS, kmajor(sK), slot(0), dS, false);
        mma_commit(lead, bS);
        mma_kk<DP, kHalf, kHalf>(lead, tDp, kmajor(sV), slot(1), dS, false);
        mma_commit(lead, bDp);
      }
      for (int u = 0; ok && u < n; ++u) {
        if (!(ok = warp_wait(bP, u & 1, stop))) break;
        fence_after();
        second(tDv, tS, slot_mn(2 * u + 1), u > 0);
        if (u + 1 < n) {
          if (!(ok = full(2 * u + 2))) break;
          mma_kk<DP, kHalf, kHalf>(lead, tS, kmajor(sK), slot(2 * u + 2), dS, false);
          mma_commit(lead, bS);
        }
        if (!(ok = warp_wait(bDs, u & 1, stop))) break;
        fence_after();
        second(tDk, tDp, slot_mn(2 * u), u > 0);
        if (TWO) second(tDk, tDp + 32, slot_mn(2 * u), true);
        mma_commit(lead, bEmpty + 8 * (2 * u % NS));
        mma_commit(lead, bEmpty + 8 * ((2 * u + 1) % NS));
        if (u + 1 < n) {
          if (!(ok = full(2 * u + 3))) break;
          mma_kk<DP, kHalf, kHalf>(lead, tDp, kmajor(sV), slot(2 * u + 3), dS, false);
          mma_commit(lead, bDp);
        }
      }
      mma_commit(lead, bEnd);
    }
  } else {
    // ---- P and dS: key r of the tile in lane r, 64 query columns a warpgroup
    const int w = warp / 4, r = tid - 128 * w;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const int64_t j = g.t0 + r;
    const int64_t jlo = g.t0 + (warp % 4) * 32, jhi = jlo + 31;  // the warp's keys
    const bool first = j < a.S;
    bool ok = true;
    // The queries' statistics, one of each a tile: warpgroup 0 brings the next tile's
    // lse as soon as every warp has P, warpgroup 1 this tile's delta once dS of the
    // last is done, both from loads that were issued a tile earlier.
    int hh = n > 0 ? u0 / per : 0, tt = n > 0 ? u0 % per : 0;  // head and query tile of the next load
    const auto fetch = [&](bool some) {
      const int64_t row = (lo + tt) * kRows + r;
      const bool on = some && row < g.nq;
      const int64_t at = ((int64_t)b * a.Hq + hk * a.G + hh) * a.Tq + g.qbeg + row;
      if (++tt == per) tt = 0, ++hh;
      if (w == 0) return on ? a.lse[at] * 1.44269504088896341f : INFINITY;  // past the sequence: p = 0
      return on ? a.delta[at] : 0.f;
    };
    float stat = fetch(n > 0);
    if (w == 0 && n > 0) {
      s_lse[r] = stat;
      __syncwarp();
      if (lane == 0) bar_arrive(bLse);
      __syncwarp();
      stat = fetch(n > 1);
    }
    int64_t t0 = (lo + (n > 0 ? u0 % per : 0)) * kRows;  // first query row of the tile
    for (int u = 0; u < n; ++u, t0 = t0 + kRows == (lo + per) * kRows ? lo * kRows : t0 + kRows) {
      const int64_t p0 = g.off + t0 + 64 * w;  // first position of the columns
      if (!(ok = warp_wait(bLse, u & 1, stop))) break;
      if (!(ok = warp_wait(bS, u & 1, stop))) break;
      fence_after();
      uint32_t s[2][32];
      tmem_ld32(tS + lanes + 64 * w, s[0]);
      tmem_ld32(tS + lanes + 64 * w + 32, s[1]);
      ld_wait();
      // columns [lo, hi] see key j
      const bool whole = jhi <= p0 && (p0 + 63 - jlo < a.W || jhi < a.S) && t0 + 64 * w + 63 < g.nq;
      if (whole) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 32; ++c)
            s[i][c] = __float_as_uint(
                fast_exp2(fmaf(__uint_as_float(s[i][c]), a.sl2, -s_lse[64 * w + 32 * i + c])));
      } else {
        const int64_t left = g.nq - t0 - 64 * w - 1;
        int64_t z = first ? 63 : j + a.W - 1 - p0;
        z = z < left ? z : left;
        const int lo_c = (int)(j - p0 < -1 ? -1 : j - p0 > 64 ? 64 : j - p0), hi_c = (int)(z < -1 ? -1 : z > 63 ? 63 : z);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int x = 32 * i + c;
            const float e = fast_exp2(fmaf(__uint_as_float(s[i][c]), a.sl2, -s_lse[64 * w + x]));
            s[i][c] = x >= lo_c && x <= hi_c ? __float_as_uint(e) : 0u;
          }
      }
      {
        // P and, below, dS go to the products as bf16, the type that the tensor cores take
        // next to bf16 operands: off by 2^-9 of themselves at most (TWO: dS as two parts, off
        // by 2^-18). dS is formed from the P of 32 bits, and all sums are of 32 bits.
        uint32_t o[32];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 16; ++c)
            o[16 * i + c] = pack_bf16(__uint_as_float(s[i][2 * c]), __uint_as_float(s[i][2 * c + 1]));
        tmem_st32(tS + lanes + 64 * w, o);
      }
      const int past = a.cu && t0 + kRows > g.nq ? (int)(g.nq - t0) : kRows;
      if (past < kRows) {  // rows of the next sequence
        const int sl = (2 * u + 1) % NS;
        if (!(ok = warp_wait(bFull + 8 * sl, ((2 * u + 1) / NS) & 1, stop))) break;
        clear_rows<DP>(sR + sl * P::kTileBytes, past, tid);
      }
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bP);
      if (w == 0 && u + 1 < n) {
        if (!(ok = warp_wait(bP, u & 1, stop))) break;
        s_lse[r] = stat;
        __syncwarp();
        if (lane == 0) bar_arrive(bLse);
        stat = fetch(u + 2 < n);
      }
      if (w == 1) {
        if (u > 0 && !(ok = warp_wait(bDs, (u - 1) & 1, stop))) break;
        s_delta[r] = stat;
        __syncwarp();
        if (lane == 0) bar_arrive(bDelta);
        stat = fetch(u + 1 < n);
      }
      if (!(ok = warp_wait(bDelta, u & 1, stop))) break;
      if (!(ok = warp_wait(bDp, u & 1, stop))) break;
      fence_after();
      uint32_t o[32], rest[TWO ? 32 : 1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t d[32];
        tmem_ld32(tDp + lanes + 64 * w + 32 * i, d);
        ld_wait();
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float e[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p = __uint_as_float(s[i][c + y]);
            const float v = p * (__uint_as_float(d[c + y]) - s_delta[64 * w + 32 * i + c + y]);
            e[y] = whole || p != 0.f ? v : 0.f;  // what lies outside may be anything
          }
          o[16 * i + c / 2] = pack_bf16(e[0], e[1]);
          if (TWO) rest[16 * i + c / 2] = rest_bf16(o[16 * i + c / 2], e[0], e[1]);
        }
      }
      tmem_st32(tDp + lanes + 64 * w, o);
      if constexpr (TWO) tmem_st32(tDp + lanes + 64 * w + 32, rest);
      if (past < kRows) clear_rows<DP>(sR + (2 * u % NS) * P::kTileBytes, past, tid);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bDs);
    }
    if (ok && n > 0) ok = warp_wait(bEnd, 0, stop);
    if (__all_sync(0xffffffffu, ok)) {
      // ---- warpgroup 0 writes dv, warpgroup 1 dk
      fence_after();
      const uint32_t sum = (w == 0 ? tDv : tDk) + lanes;
      const float f = w == 0 ? 1.f : a.scale;
      const bool live = j < g.nk;
      if (piece >= 0) {
        float* out = a.part + ((((int64_t)(b * a.Hk + hk) * a.pieces + piece) * a.sink_tiles + tile) * 2 + w) * kRows * a.D +
                     (int64_t)r * a.D;
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(sum + 32 * i, o);
            ld_wait();
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            if (32 * i + c < a.D)
              *reinterpret_cast<float4*>(out + 32 * i + c) =
                  n > 0 ? make_float4(f * __uint_as_float(o[c]), f * __uint_as_float(o[c + 1]),
                                      f * __uint_as_float(o[c + 2]), f * __uint_as_float(o[c + 3]))
                        : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else {
        __nv_bfloat16* const out = w == 0 ? a.dvp + b * a.dv_sb + (g.kbeg + j) * a.dv_st + hk * a.dv_sh
                                          : a.dkp + b * a.dk_sb + (g.kbeg + j) * a.dk_st + hk * a.dk_sh;
        if (n == 0) {  // no query sees these keys
          if (live)
            for (int c = 0; c < a.D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
        } else {
          const bool direct = a.cu && g.t0 + kRows > g.nk;
          const uint32_t so = w == 0 ? sV : sK;
          write_row<DP>(sum, f, so, r, direct, live, out, a.D);
          if (!direct) {
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bOut + 8 * w);
            if (r == 0 && bar_wait(bOut + 8 * w, 0, stop)) {
#pragma unroll
              for (int i = 0; i < DP / 64; ++i)
                copy_out_4d(w == 0 ? &a.dv : &a.dk, so + i * kHalf, 64 * i, hk, (int)(g.kbeg + g.t0), b);
              copy_out_commit();
              copy_out_done();
            }
          }
        }
      }
    }
  }
  __syncwarp();
  linger(stop);
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    tmem_free(tm, 512);
  }
}

// Adds the pieces of the cut key tiles in order: one block a (batch row and head,
// sink tile, key), dk and dv.
__global__ void __launch_bounds__(256) window_pieces_kernel(const __grid_constant__ BwdArgs a) {
  const int64_t bh = blockIdx.y;
  const int b = (int)(bh / a.Hk), hk = (int)(bh % a.Hk);
  const int64_t j = blockIdx.x, tile = j / kRows;
  if (j >= a.Tk) return;
  for (int i = threadIdx.x; i < 2 * a.D; i += 256) {
    const int w = i / a.D, c = i % a.D;
    const int64_t step = (int64_t)a.sink_tiles * 2 * kRows * a.D;
    const float* p = a.part + (bh * a.pieces * a.sink_tiles + tile) * 2 * kRows * a.D +
                     ((int64_t)w * kRows + j % kRows) * a.D + c;
    float s = 0.f;
    for (int x = 0; x < a.pieces; ++x) s += p[x * step];
    __nv_bfloat16* out = w == 0 ? a.dvp + b * a.dv_sb + j * a.dv_st + hk * a.dv_sh
                                : a.dkp + b * a.dk_sb + j * a.dk_st + hk * a.dk_sh;
    out[c] = __float2bfloat16_rn(s);
  }
}

// ---------------------------------------------------------------------------

template <int DP, bool TWO>
__global__ void __launch_bounds__(kThreadsDq, 1) window_dq_kernel(const __grid_constant__ BwdArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t sQ = base, sD = base + P::kTileBytes, sR = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bQ = bars, bFull = bars + 8, bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS, bDp = bS + 16,
                 bDs = bDp + 8, bEnd = bDs + 8 * kDsBarriers, bOut = bEnd + 8, bRow = bOut + 8;
  uint32_t* const tmem_ptr = misc + 64;
  uint32_t* const stop_flag = misc + 65;
  float* const s_row = reinterpret_cast<float*>(misc + 72);  // a row's sum of p dP, of each half of the columns

  TileRows g;
  if (!tile_rows(a.cu, a.n_seqs, a.Tq, a.Tk, blockIdx.x, kRows, &g)) return;
  const int h = blockIdx.y % a.Hq, hk = h / a.G, b = blockIdx.y / a.Hq;
  const int64_t rows = g.nq - g.t0 < kRows ? g.nq - g.t0 : kRows;
  const KeyTiles kt = key_tiles(g.off + g.t0, g.off + g.t0 + rows - 1, g.nk, a.W, a.S, kRows);
  const int n = (int)kt.count();

  // keys (u even) or values of tile u / 2 into their slot
  const auto load = [&](int u) {
    const int sl = u % NS, t = (int)(g.kbeg + kt.at(u / 2) * kRows);
    bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
    for (int i = 0; i < DP / 64; ++i)
      copy_in_4d(sR + sl * P::kTileBytes + i * kHalf, u & 1 ? &a.v : &a.k, bFull + 8 * sl, 64 * i, hk, t, b);
  };
  // the copy warp sets the barriers up and starts the first copies while the others prepare
  if (warp == 8 && lane == 0) {
    *stop_flag = 0;
    bar_init(bQ, 1);
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 1);
    }
    bar_init(bS, 1);
    bar_init(bS + 8, 1);
    bar_init(bDp, 1);
    for (int i = 0; i < kDsBarriers; ++i) bar_init(bDs + 8 * i, 8);
    bar_init(bEnd, 1);
    bar_init(bOut, 4);
    bar_init(bRow, 8);
    bar_init_fence();
    if (n > 0) {
      bar_expect(bQ, 2 * P::kTileBytes);
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        copy_in_4d(sQ + i * kHalf, &a.q, bQ, 64 * i, h, (int)(g.qbeg + g.t0), b);
        copy_in_4d(sD + i * kHalf, &a.dout, bQ, 64 * i, h, (int)(g.qbeg + g.t0), b);
      }
      for (int u = 0; u < NS && u < 2 * n; ++u) load(u);
    }
  }
  __syncwarp();
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *tmem_ptr, tS = tm, tDp = tm + 256, tDq = tm + 384;  // two S tiles
  const Stop stop{stop_flag, a.hdr};

  if (warp == 8) {
    if (lane == 0) {
      for (int u = NS; u < 2 * n; ++u) {
        if (!bar_wait(bEmpty + 8 * (u % NS), (u / NS - 1) & 1, stop)) break;
        load(u);
      }
    }
  } else if (warp == 9) {
    // ---- products: S and dq += dS k
    if (n > 0) {
      const bool lead = lane == 0;
      constexpr uint32_t dS = product_desc(128, 128, false, false);
      constexpr uint32_t dO = product_desc(128, DP, false, true);
      const auto slot = [&](int u) { return (u % NS) * (P::kTileBytes >> 4); };
      const auto full = [&](int u) { return warp_wait(bFull + 8 * (u % NS), (u / NS) & 1, stop); };
      const auto scores = [&](int u) {
        mma_kk<DP, kHalf, kHalf>(lead, tS + 128 * (u & 1), kmajor(sQ), kmajor(sR) + slot(2 * u), dS, false);
        mma_commit(lead, bS + 8 * (u & 1));
      };
      bool ok = warp_wait(bQ, 0, stop) && full(0);
      if (ok) scores(0);
      if (ok && n > 1 && (ok = full(2))) scores(1);
#pragma unroll 1
      for (int u = 0; ok && u < n; ++u) {
        if (!(ok = warp_wait(bDs + 8 * ds_barrier(u), ds_parity(u), stop))) break;
        fence_after();
        const uint32_t w = tS + 128 * (u & 1), t = mnmajor(sR, kHalf) + slot(2 * u);
        mma_tn<64>(lead, tDq, w, t, dO, u > 0);
        mma_tn<64>(lead, tDq, w + 64, t + (64 * kPitch >> 4), dO, true);
        if (TWO) {
          mma_tn<64>(lead, tDq, w + 32, t, dO, true);
          mma_tn<64>(lead, tDq, w + 96, t + (64 * kPitch >> 4), dO, true);
        }
        mma_commit(lead, bEmpty + 8 * (2 * u % NS));
        if (u + 2 < n) {
          if (!(ok = full(2 * u + 4))) break;
          scores(u + 2);
        }
      }
      mma_commit(lead, bEnd);
    }
  } else if (warp == 10) {
    // ---- products: dP
    if (n > 0) {
      const bool lead = lane == 0;
      constexpr uint32_t dS = product_desc(128, 128, false, false);
      bool ok = warp_wait(bQ, 0, stop);
#pragma unroll 1
      for (int u = 0; ok && u < n; ++u) {
        const int v = (2 * u + 1) % NS;
        if (!(ok = warp_wait(bFull + 8 * v, ((2 * u + 1) / NS) & 1, stop))) break;
        if (u > 0 && !(ok = warp_wait(bDs + 8 * ds_barrier(u - 1), ds_parity(u - 1), stop))) break;  // the last dP has been read
        fence_after();
        mma_kk<DP, kHalf, kHalf>(lead, tDp, kmajor(sD), kmajor(sR) + v * (P::kTileBytes >> 4), dS, false);
        mma_commit(lead, bDp);
        mma_commit(lead, bEmpty + 8 * v);
      }
    }
  } else {
    const int w = warp / 4, r = tid - 128 * w;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const int64_t row = g.t0 + r, pos = g.off + row;
    const int64_t wlo = g.off + g.t0 + (warp % 4) * 32, whi = wlo + 31;
    const bool live = row < g.nq;
    const int64_t at = ((int64_t)b * a.Hq + h) * a.Tq + g.qbeg + row;
    const float lse = live ? a.lse[at] * 1.44269504088896341f : INFINITY;
    float delta = live && n > 1 ? a.delta[at] : 0.f;
    bool ok = true;
    for (int u = 0; u < n; ++u) {
      const int64_t j0 = kt.at(u) * kRows, c0 = j0 + 64 * w;  // first key of the columns
      if (!(ok = warp_wait(bS + 8 * (u & 1), (u >> 1) & 1, stop))) break;
      fence_after();
      uint32_t s[2][32];
      tmem_ld32(tS + 128 * (u & 1) + lanes + 64 * w, s[0]);
      tmem_ld32(tS + 128 * (u & 1) + lanes + 64 * w + 32, s[1]);
      ld_wait();
      const bool whole = c0 + 63 <= wlo && (whi - c0 < a.W || c0 + 64 <= a.S) && g.t0 + (warp % 4) * 32 + 31 < g.nq;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 32; ++c)
          s[i][c] = __float_as_uint(fast_exp2(fmaf(__uint_as_float(s[i][c]), a.sl2, -lse)));
      if (!whole) {
        const auto cl = [](int64_t v) { return (int)(v < -1 ? -1 : v > 64 ? 64 : v); };
        const int lo = cl(pos - a.W + 1 - c0), hi = live ? cl(pos - c0) : -1, sk = cl(a.S - c0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int x = 32 * i + c;
            if (!(x <= hi && (x >= lo || x < sk))) s[i][c] = 0u;
          }
      }
      if (!(ok = warp_wait(bDp, u & 1, stop))) break;
      fence_after();
      if (n == 1) {
        // The row's weights are all here, so delta = do o = sum p dP is formed from them, in
        // 32 bits: where keys are few, one from the output as it was rounded is a large part
        // of the error. The keys' kernel, which comes after, reads it.
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t d[32];
          tmem_ld32(tDp + lanes + 64 * w + 32 * i, d);
          ld_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float p = __uint_as_float(s[i][c]);
            if (whole || p != 0.f) sum = fmaf(p, __uint_as_float(d[c]), sum);
          }
        }
        s_row[128 * w + r] = sum;
        __syncwarp();
        if (lane == 0) bar_arrive(bRow);
        if (!(ok = warp_wait(bRow, 0, stop))) break;
        delta = s_row[r] + s_row[128 + r];
        if (w == 0 && live) a.delta[at] = delta;
      }
      uint32_t o[32], rest[TWO ? 32 : 1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t d[32];
        tmem_ld32(tDp + lanes + 64 * w + 32 * i, d);
        ld_wait();
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          float e[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p = __uint_as_float(s[i][c + y]);
            const float v = p * (__uint_as_float(d[c + y]) - delta);
            e[y] = whole || p != 0.f ? v : 0.f;
          }
          // (one bf16 part or two, as in the keys' kernel)
          o[16 * i + c / 2] = pack_bf16(e[0], e[1]);
          if (TWO) rest[16 * i + c / 2] = rest_bf16(o[16 * i + c / 2], e[0], e[1]);
        }
      }
      tmem_st32(tS + 128 * (u & 1) + lanes + 64 * w, o);
      if constexpr (TWO) tmem_st32(tS + 128 * (u & 1) + lanes + 64 * w + 32, rest);
      if (a.cu && j0 + kRows > g.nk)  // key rows of the next sequence (its scores are done)
        clear_rows<DP>(sR + (2 * u % NS) * P::kTileBytes, (int)(g.nk - j0), tid);
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bDs + 8 * ds_barrier(u));
    }
    if (ok && n > 0) ok = warp_wait(bEnd, 0, stop);
    if (w == 0 && __all_sync(0xffffffffu, ok)) {
      fence_after();
      __nv_bfloat16* const out = a.dqp + b * a.dq_sb + (g.qbeg + row) * a.dq_st + h * a.dq_sh;
      if (n == 0) {  // these queries see nothing
        if (live)
          for (int c = 0; c < a.D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
      } else {
        const bool direct = a.cu && g.t0 + kRows > g.nq;
        write_row<DP>(tDq + lanes, a.scale, sQ, r, direct, live, out, a.D);
        if (!direct) {
          fence_async();
          __syncwarp();
          if (lane == 0) bar_arrive(bOut);
          if (r == 0 && bar_wait(bOut, 0, stop)) {
#pragma unroll
            for (int i = 0; i < DP / 64; ++i)
              copy_out_4d(&a.dq, sQ + i * kHalf, 64 * i, h, (int)(g.qbeg + g.t0), b);
            copy_out_commit();
            copy_out_done();
          }
        }
      }
    }
  }
  __syncwarp();
  linger(stop);
  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    tmem_free(tm, 512);
  }
}

template <int DP, bool TWO>
cudaError_t launch_bwd(const BwdArgs& t, int64_t B, cudaStream_t s) {
  using P = Plan<DP>;
  static_assert(P::kSmem <= 232448, "fits a block's shared memory");
  cudaError_t e = cudaFuncSetAttribute(window_dkv_kernel<DP, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(window_dq_kernel<DP, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t extra = t.cu ? t.n_seqs : 0;
  const int64_t tk = (t.Tk + kRows - 1) / kRows + extra, tq = (t.Tq + kRows - 1) / kRows + extra;
  const int64_t cut = t.pieces > 1 ? (int64_t)t.sink_tiles * (t.pieces - 1) : 0;
  window_dq_kernel<DP, TWO><<<dim3((unsigned)tq, (unsigned)(B * t.Hq)), kThreadsDq, P::kSmem, s>>>(t);
  window_dkv_kernel<DP, TWO><<<dim3((unsigned)(tk + cut), (unsigned)(B * t.Hk)), kThreads, P::kSmem, s>>>(t);
  if (t.pieces > 1)
    window_pieces_kernel<<<dim3((unsigned)(t.sink_tiles * kRows), (unsigned)(B * t.Hk)), 256, 0, s>>>(t);
  return cudaGetLastError();
}

// The walk of a key tile that holds first tokens, in pieces no longer than any
// other tile's walk (dense rows; at most 64 pieces, and 16 cut tiles).
struct Cut {
  int tiles, pieces;
};
Cut cut_sinks(int64_t Tq, int64_t Tk, int64_t W, int64_t S, bool packed) {
  if (packed || S < 1 || Tk < 1) return Cut{0, 1};
  const int64_t all = (Tq + kRows - 1) / kRows, one = (W + 2 * kRows - 2) / kRows + 1;
  const int64_t tiles = ((S < Tk ? S : Tk) + kRows - 1) / kRows;
  int64_t p = (all + one - 1) / one;
  if (p > 64) p = 64;
  if (p < 2 || tiles > 16) return Cut{0, 1};
  return Cut{(int)tiles, (int)p};
}

// Whether dS goes to its products as the sum of two bf16 parts. Past its first tile of
// keys a row's delta comes from the output as it was rounded, which is felt where it sees
// few keys (an error of (keys / e - 1)^(-1/2) roundings for scores of unit variance):
// together with the rounding of dS it would be more than the gradients' own. Short rows,
// and narrow windows, so take the two parts; elsewhere one rounding is what is left. Error
// of dq and dk in the 2-norm (with delta from the rounded output everywhere) and us of the
// backward, one part / two, 16 heads of 128 over 4: 4 x 64 tokens 2.6e-3 / 2.0e-3, 24 / 26
// us; 2 x 512 2.5e-3 / 1.9e-3, 48 / 55 us; 2 x 4096, window 1024 2.4e-3 / 1.8e-3, 302 / 346
// us (rounding the exact gradients alone: 1.7e-3).
bool two_parts(const WinArgs& a) {
  const int64_t len = a.cu ? a.Tk / a.n_seqs : a.Tk;  // of a sequence, in the mean
  return len <= 512 || a.W + a.S <= 64;
}

}  // namespace

size_t window_tc_bwd_floats(int64_t B, int64_t Tq, int64_t Tk, int64_t Hk, int64_t D, int64_t W, int64_t S,
                            bool packed) {
  const Cut c = cut_sinks(Tq, Tk, W, S, packed);
  return c.pieces < 2 ? 0 : (size_t)(B * Hk * c.pieces * c.tiles) * 2 * kRows * (size_t)D;
}

cudaError_t launch_window_tc_bwd(const WinArgs& a, float* part, cudaStream_t s) {
  BwdArgs t;
  if (!encode_heads_map(&t.q, a.q, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.k, a.k, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.v, a.v, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.dout, a.dout, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.dq, a.dq, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.dk, a.dk, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.dv, a.dv, a.B, a.Tk, a.Hk, a.D, kRows))
    return cudaErrorInvalidValue;
  t.dqp = static_cast<__nv_bfloat16*>(a.dq.ptr);
  t.dq_sb = a.dq.stride_b, t.dq_st = a.dq.stride_t, t.dq_sh = a.dq.stride_h;
  t.dkp = static_cast<__nv_bfloat16*>(a.dk.ptr);
  t.dk_sb = a.dk.stride_b, t.dk_st = a.dk.stride_t, t.dk_sh = a.dk.stride_h;
  t.dvp = static_cast<__nv_bfloat16*>(a.dv.ptr);
  t.dv_sb = a.dv.stride_b, t.dv_st = a.dv.stride_t, t.dv_sh = a.dv.stride_h;
  t.lse = a.lse;
  t.delta = a.delta;
  t.part = part;
  t.cu = a.cu;
  t.hdr = a.hdr;
  t.Tq = a.Tq;
  t.Tk = a.Tk;
  t.W = a.W;
  t.S = a.S;
  t.n_seqs = a.n_seqs;
  t.Hq = a.Hq;
  t.Hk = a.Hk;
  t.G = a.Hq / a.Hk;
  t.D = a.D;
  DeltaArgs d;
  d.o = static_cast<const __nv_bfloat16*>(a.o.ptr);
  d.o_sb = a.o.stride_b, d.o_st = a.o.stride_t, d.o_sh = a.o.stride_h;
  d.d = static_cast<const __nv_bfloat16*>(a.dout.ptr);
  d.d_sb = a.dout.stride_b, d.d_st = a.dout.stride_t, d.d_sh = a.dout.stride_h;
  d.delta = a.delta;
  d.T = a.Tq;
  d.H = a.Hq;
  d.D = a.D;
  d.rows = a.B * a.Tq * a.Hq;
  window_delta16_kernel<<<(unsigned)((d.rows + 63) / 64), 256, 0, s>>>(d);
  const Cut c = cut_sinks(a.Tq, a.Tk, a.W, a.S, a.cu != nullptr);
  t.sink_tiles = c.tiles;
  t.pieces = c.pieces;
  t.sl2 = a.scale * 1.44269504088896341f;
  t.scale = a.scale;
  const bool two = two_parts(a);
  if (a.D <= 64) return two ? launch_bwd<64, true>(t, a.B, s) : launch_bwd<64, false>(t, a.B, s);
  return two ? launch_bwd<128, true>(t, a.B, s) : launch_bwd<128, false>(t, a.B, s);
}

}  // namespace scan
