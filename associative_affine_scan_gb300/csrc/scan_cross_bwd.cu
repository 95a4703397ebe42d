// scan_cross_bwd.cu -- backward of attention to another sequence, on the tensor cores
// (bf16 operands).
//
//   p = 2^(scale log2(e) q k - lse log2(e)), ds = p (do v - delta), delta = do o
//   dv = sum p do, dk = scale sum ds q (over queries and the heads that share the
//   key head), dq = scale sum ds k (over keys)
//
// Two kernels, each with its sums in tensor memory: the five products become seven, but
// nothing is added in global memory in an order that changes.
//   queries: a block takes tiles of 128 queries of a head, one after the other, and walks
//            the key tiles: S = q k^T, dP = do v^T, dq += dS k. It runs first: where the
//            queries see one tile of keys, it forms their delta anew from p and dP, for
//            the keys' kernel as well.
//   keys:    tiles of 128 keys against the tiles of 128 queries of the heads that share
//            them: S = k q^T, dP = v do^T, dv += P do, dk += dS q. Keys are the rows of S,
//            so P and dS (bf16, over S and dP in tensor memory) are read as they lie by the
//            second products. Encoders have few tiles of keys, each with many queries: the
//            (key tile, query tile) pairs are dealt out in order to one block an SM, equal
//            shares of the work each. A key tile that a share's end cuts leaves its parts in the
//            workspace (at most two a block), which a last kernel adds in order.
// Either kernel issues the products of its two chains from two warps, so that one's waits
// and commits are under the other's products.
//
// 4 x 4096 queries over 1280 to 2048 keys, 16 heads of 128 over 4: row sums 25 us (DRAM, 5.4
// TB/s), queries 249 us (three products, 1.34 PFLOP/s), keys 348 us (four, 1.29 PFLOP/s),
// parts 12 us.
// Bound by a pair of tiles' chain: the softmax of S, dS from dP, and their handing over and
// back leave the tensor cores idle for a quarter to a third of the time. Shorter rows are
// bound by the tiles' beginnings and ends (seven packed sequences of 46 to 1314 keys, 12
// heads of 96: row sums 8 us, queries 42 us, keys 57 us, parts 8 us; with dS of the short ones
// in one part queries 40 us, keys 52 us).
#include "scan_cross_phases.h"
#include "scan_cross_tc.h"
#include "scan_tc.cuh"

namespace scan {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kThreads = 12 * 32;  // two warpgroups of softmax; copies, two of products, row statistics
constexpr uint32_t kHalf = kRows * kPitch;
constexpr int kBlocks = 152;  // one an SM

// A key tile that is cut: what the block whose share it begins in leaves for the last kernel.
struct Cut {
  int32_t parts;  // blocks that have parts of it; 0: none
  int32_t b, hk, live;
  int64_t key;    // its first key row, and how many of its rows have gradients
  int64_t rows;   // and how many are written
};

struct BwdArgs {
  CUtensorMap q, k, v, dout;
  __nv_bfloat16 *dqp, *dkp, *dvp;
  int64_t dq_sb, dq_st, dq_sh, dk_sb, dk_st, dk_sh, dv_sb, dv_st, dv_sh;
  const float* lse;
  float* delta;
  float* part;  // [blocks][2][2][D / 4][128][4]: a block's cut tiles, the first and the last; dv and dk
  Cut* cut;     // [blocks]
  const int32_t *lens, *cu_q, *cu_k;
  WsHeader* hdr;
  int64_t B, Tq, Tk;
  int64_t tiles, items;  // query tiles of a (batch row, head), and of all
  int n_seqs, Hq, Hk, G, D;
  int order;          // query tiles: the longest sequences first
  int wide, wide_kv;  // rows of dq, and of dk and dv, are on 32 bytes
  float sl2, scale;
};

template <int DP>
struct Plan {
  static constexpr int kTileBytes = kRows * DP * 2;
  static constexpr int kSlots = bwd_slots(DP);
  static constexpr int kMisc = 2048;  // barriers, row statistics
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024 + kMisc;
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

// Whether dS goes to its products as the sum of two bf16 parts: its rounding to one adds as
// much to dq and dk as their own does (0.0024 of them in the 2-norm, 0.0017 with two), at any
// number of keys. The second part's products make four of the queries' kernel's three, and
// five of the keys' four. So sequences of few keys, whose pairs of tiles are a small part of
// the time, take two. By the sequence's own keys: its gradients do not depend on what else is
// in the batch, or on what that is padded to.
__device__ __forceinline__ bool two_parts(const CrossRows& g) { return g.nk <= 512; }

// d (+)= A B over 16 `steps` columns of K-major tiles, or over 64 rows of an MN-major tile
// with A in tensor memory; by the elected lane.
template <int DP>
__device__ __forceinline__ void issue_kk(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, int steps) {
#pragma unroll
  for (int c = 0; c < DP / 16; ++c) {
    if (c >= steps) break;
    const uint32_t step = (c / 4) * (kHalf >> 4) + (c % 4) * 2;
    mma_ss1(d, a + step, b + step, desc, c > 0);
  }
}
__device__ __forceinline__ void issue_tn64(uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
#pragma unroll
  for (int c = 0; c < 4; ++c) mma_ts1(d, a + 8 * c, b + c * (2048 >> 4), desc, add || c > 0);
}

// A row of D fp32 sums in tensor memory times f as bf16.
template <int DP>
__device__ __forceinline__ void write_row(uint32_t tsum, float f, bool live, bool wide, __nv_bfloat16* out, int D) {
#pragma unroll
  for (int c = 0; c < DP / 32; ++c) {
    uint32_t o[32], v[16];
    tmem_ld32(tsum + 32 * c, o);
    ld_wait();
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = pack_bf16(__uint_as_float(o[2 * j]) * f, __uint_as_float(o[2 * j + 1]) * f);
    if (live && wide) {
      if (32 * c < D) st_global32(out + 32 * c, v);
      if (32 * c + 16 < D) st_global32(out + 32 * c + 16, v + 8);
    } else if (live) {
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        if (32 * c + 2 * j < D)
          *reinterpret_cast<uint4*>(out + 32 * c + 2 * j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  }
}
__device__ __forceinline__ void zero_row(bool live, __nv_bfloat16* out, int D) {
  if (live)
    for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------

struct DeltaArgs {
  const __nv_bfloat16 *o, *d;
  int64_t o_sb, o_st, o_sh, d_sb, d_st, d_sh;
  float* delta;
  int64_t T, rows;
  int H, D;
};

// delta = sum of dout o of every row: 16 lanes of 16 bytes a row, four rows in flight a
// lane. Bound by DRAM.
__global__ void __launch_bounds__(256) cross_delta_kernel(const DeltaArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
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

// ---------------------------------------------------------------------------
// queries

// A tile of queries of head h.
struct Item {
  CrossRows g;
  int b, h, hk;
  int n;  // tiles of keys
};
__device__ __forceinline__ bool item_at(const BwdArgs& a, const Order& order, int64_t i, Item* w) {
  if (a.order) {
    int64_t unit, tile;
    int s;
    if (!order.find(i, a.Hq, &s, &unit, &tile)) return false;
    w->g = rows_of(a.lens, a.cu_q, a.cu_k, a.Tq, a.Tk, s, tile * kRows);
    w->b = a.cu_q ? 0 : s;
    w->h = (int)unit;
    w->hk = w->h / a.G;
    w->n = (int)((w->g.nk + kRows - 1) / kRows);
    return true;
  }
  const int64_t unit = i / a.tiles, tile = i - unit * a.tiles;
  w->b = (int)(unit / a.Hq);
  w->h = (int)(unit % a.Hq);
  w->hk = w->h / a.G;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, w->b, tile, kRows, false, &w->g)) return false;
  w->n = (int)((w->g.nk + kRows - 1) / kRows);
  return true;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) cross_dq_kernel(const __grid_constant__ BwdArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = (int)uniform(tid / 32), lane = tid % 32;
  const int steps = (a.D + 15) / 16;  // what D leaves of the DP columns is neither multiplied nor summed
  const uint32_t sQ = base, sD = base + P::kTileBytes, sR = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bQ = bars, bD = bars + 8, bQfree = bars + 16, bDfree = bars + 24, bFull = bars + 32,
                 bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS, bDp = bS + 16, bRead = bDp + 8, bDs = bRead + 8,
                 bEnd = bDs + 16, bRow = bEnd + 8;
  uint32_t* const tmem_ptr = misc + 64;
  uint32_t* const stop_flag = misc + 65;
  float* const s_row = reinterpret_cast<float*>(misc + 72);  // a row's sum of p dP, of each half of the columns
  Order& order = *reinterpret_cast<Order*>(misc + 332);

  if (warp == 8 && lane == 0) {
    *stop_flag = 0;
    bar_init(bQ, 1);
    bar_init(bD, 1);
    bar_init(bQfree, 1);
    bar_init(bDfree, 1);
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 1);
    }
    bar_init(bS, 1);
    bar_init(bS + 8, 1);
    bar_init(bDp, 1);
    bar_init(bRead, 8);
    // Two barriers for dS by turns: dS of the next tile can be made before the product warp
    // has seen this one's, but that of the one after needs scores which it issues later.
    bar_init(bDs, 8);
    bar_init(bDs + 8, 8);
    bar_init(bEnd, 1);
    bar_init(bRow, 8);
    bar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  if (a.order && warp == 10)
    order.make(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, kRows, a.Hq);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(*tmem_ptr), tS = tm, tDp = tm + 256, tDq = tm + 384;  // two S tiles
  const Stop stop{stop_flag, a.hdr};
  bool ok = true;
  asm volatile("griddepcontrol.launch_dependents;");
  Item w;
  const auto full = [&](uint32_t c) { return warp_wait(bFull + 8 * (c % NS), (c / NS) & 1, stop); };
  // the next item with keys
  int64_t round = 0;
  const auto next_item = [&]() {
    for (; item_of(round, a.order) < a.items; ++round)
      if (item_at(a, order, item_of(round, a.order), &w) && w.n > 0) break;
    const bool some = __any_sync(0xffffffffu, item_of(round, a.order) < a.items);
    ++round;
    return some;
  };

  if (warp == 8) {
    // ---- copies: queries and output gradients, and keys (kv even) and values by turns
    uint32_t kv = 0, seen = 0;
    while (ok && next_item()) {
      if (lane == 0) {
        const auto load = [&](int u) {
          const uint32_t sl = kv % NS;
          if (kv >= NS && !bar_wait(bEmpty + 8 * sl, (kv / NS - 1) & 1, stop)) return false;
          bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            copy_in_4d(sR + sl * P::kTileBytes + c * kHalf, u & 1 ? &a.v : &a.k, bFull + 8 * sl, 64 * c, w.hk,
                       (int)(w.g.kbeg + (int64_t)(u / 2) * kRows), w.b);
          ++kv;
          return true;
        };
        const auto rows = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t free) {
          if (seen > 0 && !bar_wait(free, (seen - 1) & 1, stop)) return false;
          bar_expect(bar, P::kTileBytes);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            copy_in_4d(dst + c * kHalf, map, bar, 64 * c, w.h, (int)(w.g.qbeg + w.g.t0), w.b);
          return true;
        };
        ok = load(0) && rows(sQ, &a.q, bQ, bQfree) && load(1) && rows(sD, &a.dout, bD, bDfree);
        for (int u = 2; ok && u < 2 * w.n; ++u) ok = load(u);
      }
      ++seen;
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp == 9) {
    // ---- products: S, two tiles ahead, and dq += dS k
    constexpr uint32_t dS = product_desc(128, 128, false, false);
    const uint32_t dO = product_desc(128, 16 * steps, false, true);
    uint32_t s = 0, items = 0;  // scores issued, items begun
    int left = 0;               // tiles of the current item whose scores are to come
    bool more = true;
    // scores of the next tile, of this item or the next; and how many tiles of an item were left
    const auto scores = [&]() {
      if (left == 0) {
        if (!(more = next_item())) return;
        left = (int)uniform(w.n);
        if (!(ok = warp_wait(bQ, items & 1, stop))) return;
        ++items;
      }
      if (!(ok = full(2 * s))) return;
      const uint32_t k = uniform(kmajor(sR) + (2 * s % NS) * (P::kTileBytes >> 4)), d = tS + 128 * (s & 1);
      if (elect()) {
        issue_kk<DP>(d, kmajor(sQ), k, dS, steps);
        commit1(bS + 8 * (s & 1));
      }
      __syncwarp();
      --left;
      ++s;
    };
    // which tiles begin and end an item: a second walk, two tiles behind
    int64_t back_round = 0;
    Item bw;
    int back_left = 0;
    bool two = false;
    scores();
    if (ok && more) scores();
    for (uint32_t t = 0; ok && t < s; ++t) {
      const bool begin = back_left == 0;
      if (begin) {
        for (; item_of(back_round, a.order) < a.items; ++back_round)
          if (item_at(a, order, item_of(back_round, a.order), &bw) && bw.n > 0) break;
        ++back_round;
        back_left = (int)uniform(bw.n);
        two = uniform(two_parts(bw.g)) != 0;
      }
      const bool end = --back_left == 0;
      const uint32_t k = uniform(mnmajor(sR, kHalf) + (2 * t % NS) * (P::kTileBytes >> 4)), d = tS + 128 * (t & 1);
      if (!(ok = warp_wait(bDs + 8 * (t & 1), (t >> 1) & 1, stop))) break;
      fence_after();
      if (elect()) {
        issue_tn64(tDq, d, k, dO, !begin);
        issue_tn64(tDq, d + 64, k + (64 * kPitch >> 4), dO, true);
        if (two) {
          issue_tn64(tDq, d + 32, k, dO, true);
          issue_tn64(tDq, d + 96, k + (64 * kPitch >> 4), dO, true);
        }
        commit1(bEmpty + 8 * (2 * t % NS));
        if (end) commit1(bEnd);
      }
      __syncwarp();
      if (more) scores();
    }
  } else if (warp == 10) {
    // ---- products: dP
    constexpr uint32_t dS = product_desc(128, 128, false, false);
    uint32_t t = 0, items = 0;
    while (ok && next_item()) {
      if (!(ok = warp_wait(bD, items & 1, stop))) break;
      ++items;
      for (int u = 0; u < w.n; ++u, ++t) {
        const uint32_t v = uniform(kmajor(sR) + ((2 * t + 1) % NS) * (P::kTileBytes >> 4));
        if (!(ok = full(2 * t + 1))) break;
        if (t > 0 && !(ok = warp_wait(bRead, (t - 1) & 1, stop))) break;  // the last dP has been read
        fence_after();
        if (elect()) {
          issue_kk<DP>(tDp, kmajor(sD), v, dS, steps);
          commit1(bDp);
        }
        __syncwarp();
      }
    }
  } else if (warp < 8) {
    // ---- dS: row r in lane r, 64 key columns a warpgroup
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for delta
    const int x = warp / 4, r = tid - 128 * x;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    uint32_t t = 0, items = 0, single = 0;
    for (int64_t round = 0; ok && item_of(round, a.order) < a.items; ++round) {
      if (!item_at(a, order, item_of(round, a.order), &w)) continue;
      const int64_t row = w.g.t0 + r;
      const bool live = row < w.g.nq;
      __nv_bfloat16* const out = a.dqp + w.b * a.dq_sb + (w.g.qbeg + row) * a.dq_st + w.h * a.dq_sh;
      if (w.n == 0) {  // no keys
        if (x == 0) zero_row(live, out, a.D);
        continue;
      }
      const int64_t st = ((int64_t)w.b * a.Hq + w.h) * a.Tq + w.g.qbeg + row;
      const float lse = live ? a.lse[st] * 1.44269504088896341f : INFINITY;
      float delta = live && w.n > 1 ? a.delta[st] : 0.f;
      const bool two = two_parts(w.g);
      for (int u = 0; u < w.n; ++u, ++t) {
        const int here = w.g.nk - (int64_t)u * kRows < kRows ? (int)(w.g.nk - (int64_t)u * kRows) : kRows;  // keys
        if (!(ok = warp_wait(bS + 8 * (t & 1), (t >> 1) & 1, stop))) break;
        fence_after();
        uint32_t s[2][32], d[2][32];
        tmem_ld32(tS + 128 * (t & 1) + lanes + 64 * x, s[0]);
        tmem_ld32(tS + 128 * (t & 1) + lanes + 64 * x + 32, s[1]);
        if (tid == 0 && u == w.n - 1) bar_arrive(bQfree);
        __syncwarp();
        ld_wait();
        const float2 sl2 = make_float2(a.sl2, a.sl2), from = make_float2(-lse, -lse);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 z = fma2(pair_of(s[c] + j), sl2, from);
            s[c][j] = __float_as_uint(fast_exp2(z.x));
            s[c][j + 1] = __float_as_uint(fast_exp2(z.y));
          }
        const bool whole = here == kRows;
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (64 * x + 32 * c + j >= here) s[c][j] = 0u;
        }
        if (!(ok = warp_wait(bDp, t & 1, stop))) break;
        fence_after();
        tmem_ld32(tDp + lanes + 64 * x, d[0]);
        tmem_ld32(tDp + lanes + 64 * x + 32, d[1]);
        if (tid == 0) {  // the products with these values are done
          bar_arrive(bEmpty + 8 * ((2 * t + 1) % NS));
          if (u == w.n - 1) bar_arrive(bDfree);
        }
        __syncwarp();
        ld_wait();
        fence_before();
        if (lane == 0) bar_arrive(bRead);
        __syncwarp();
        if (!whole) {  // what lies outside may be anything
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (64 * x + 32 * c + j >= here) d[c][j] = 0u;
        }
        if (w.n == 1) {
          // The row's weights are all here, so delta = do o = sum p dP is formed from them, in
          // 32 bits: where keys are few, one from the output as it was rounded is a large part
          // of the error. The keys' kernel, which comes after, reads it.
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) sum = fmaf(__uint_as_float(s[c][j]), __uint_as_float(d[c][j]), sum);
          s_row[128 * x + r] = sum;
          __syncwarp();
          if (lane == 0) bar_arrive(bRow);
          if (!(ok = warp_wait(bRow, single & 1, stop))) break;
          ++single;
          delta = s_row[r] + s_row[128 + r];
          if (x == 0 && live) a.delta[st] = delta;
        }
        // dS goes to its product as bf16, the type that the tensor cores take next to bf16
        // operands: off by 2^-8 of itself at most (as two parts, by 2^-16)
        uint32_t o[32];
        const float2 less = make_float2(-delta, -delta);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 e = mul2(pair_of(s[c] + j), add2(pair_of(d[c] + j), less));
            o[16 * c + j / 2] = pack_bf16(e.x, e.y);
            s[c][j] = __float_as_uint(e.x), s[c][j + 1] = __float_as_uint(e.y);
          }
        tmem_st32(tS + 128 * (t & 1) + lanes + 64 * x, o);
        if (two) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = rest_bf16(o[j], __uint_as_float(s[j / 16][2 * j % 32]), __uint_as_float(s[j / 16][2 * j % 32 + 1]));
          tmem_st32(tS + 128 * (t & 1) + lanes + 64 * x + 32, o);
        }
        if (!whole && (a.cu_q || a.lens))  // key rows past the sequence (their scores are done)
          clear_rows<DP>(sR + (2 * t % NS) * P::kTileBytes, here, tid);
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bDs + 8 * (t & 1));
        __syncwarp();
      }
      if (!ok) break;
      if (!(ok = warp_wait(bEnd, items & 1, stop))) break;
      ++items;
      fence_after();
      if (x == 0) write_row<DP>(tDq + lanes, a.scale, live, a.wide, out, a.D);
      // the next item's sums come after dS from all warps: this one's have been read by then
      fence_before();
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

// ---------------------------------------------------------------------------
// keys

// The (key tile, query tile) pairs in the order that they are dealt out: sequence by
// sequence, key head by key head, tile by tile of its keys, then of its queries over
// the heads that share them. What is dealt out in equal shares are turns: a pair is one, a
// tile's beginning and end are three more, ahead of its pairs (12 heads of 96: 1.4 us a pair,
// 4 us a beginning and end; seven packed sequences of 46 to 1314 keys, dealt out by pairs
// alone 75 us, so 52 us, dS in one part), and a tile without a pair is one.
constexpr int kEnds = 3;
struct KeyTile {
  CrossRows g;     // t0: its first key row
  int64_t first;   // its first turn
  int64_t tile;    // within the sequence and head
  int64_t tiles;   // of the sequence and head (dense: of the whole row)
  int64_t live;    // those with pairs
  int seq, hk;
  int n;           // its pairs, 0 for a tile without
  int per;         // query tiles of a head
  __device__ int64_t last() const { return first + (n > 0 ? n + kEnds : 1); }
};
// Rows, tiles and turns of sequence i.
__device__ __forceinline__ void sequence(const BwdArgs& a, int i, KeyTile* w) {
  CrossRows& g = w->g;
  if (a.cu_q) {
    int64_t qe, ke;
    seq_bounds(a.cu_q, i, a.Tq, &g.qbeg, &qe);
    seq_bounds(a.cu_k, i, a.Tk, &g.kbeg, &ke);
    g.nq = qe - g.qbeg;
    g.nk = ke - g.kbeg;
    w->tiles = (g.nk + kRows - 1) / kRows;
  } else {
    g.qbeg = g.kbeg = 0;
    g.nq = a.Tq;
    g.nk = keys_of(a.lens, i, a.Tk);
    w->tiles = (a.Tk + kRows - 1) / kRows;
  }
  w->seq = i;
  w->per = (int)((g.nq + kRows - 1) / kRows);
  w->live = g.nq > 0 ? (g.nk + kRows - 1) / kRows : 0;
}
__device__ __forceinline__ int64_t deep(const BwdArgs& a, const KeyTile& w) { return (int64_t)w.per * a.G + kEnds; }
__device__ __forceinline__ int64_t turns_of(const BwdArgs& a, const KeyTile& w) {  // of one key head
  return w.live * deep(a, w) + (w.tiles - w.live);
}
__device__ __forceinline__ void place(const BwdArgs& a, KeyTile* w) {
  w->g.t0 = w->tile * kRows;
  w->n = w->tile < w->live ? w->per * a.G : 0;
}
// The tile that holds turn `p`, or (p < 0) the number of all turns. A whole warp.
__device__ __forceinline__ int64_t find_turn(const BwdArgs& a, int64_t p, KeyTile* w) {
  const int lane = threadIdx.x & 31, n = a.cu_q ? a.n_seqs : (int)a.B;
  int64_t before = 0;
  for (int i0 = 0; i0 < n; i0 += 32) {
    int64_t mine = 0;
    if (i0 + lane < n) {
      sequence(a, i0 + lane, w);
      mine = turns_of(a, *w) * a.Hk;
    }
    int64_t upto = mine;
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const unsigned who = __ballot_sync(0xffffffffu, p >= 0 && p >= before + upto - mine && p < before + upto);
    if (who) {
      const int src = __ffs(who) - 1;
      before += __shfl_sync(0xffffffffu, upto - mine, src);
      sequence(a, i0 + src, w);
      const int64_t head = turns_of(a, *w), d = deep(a, *w);
      w->hk = (int)((p - before) / head);
      before += w->hk * head;
      const int64_t in = p - before;
      if (in < w->live * d) {
        w->tile = in / d;
        w->first = before + w->tile * d;
      } else {
        w->tile = w->live + (in - w->live * d);
        w->first = p;
      }
      place(a, w);
      return p;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return before;
}
__device__ __forceinline__ void next_tile(const BwdArgs& a, KeyTile* w) {
  w->first = w->last();
  if (++w->tile == w->tiles) {
    w->tile = 0;
    if (++w->hk == a.Hk) {
      w->hk = 0;
      do sequence(a, w->seq + 1, w);
      while (w->tiles == 0);
    }
  }
  place(a, w);
}
// How many blocks share `all` turns, and block c's first.
__device__ __forceinline__ int64_t sharers(int64_t all, int64_t blocks) {
  const int64_t n = (all + kEnds + 1) / (kEnds + 2);  // two pairs each at least
  return n < blocks ? n : blocks;
}
__device__ __forceinline__ int64_t share(int64_t all, int64_t n, int64_t c) { return all / n * c + (all % n) * c / n; }

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) cross_dkv_kernel(const __grid_constant__ BwdArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = (int)uniform(tid / 32), lane = tid % 32;
  const int steps = (a.D + 15) / 16;  // what D leaves of the DP columns is neither multiplied nor summed
  const uint32_t sK = base, sV = base + P::kTileBytes, sR = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bKV = bars, bKVfree = bars + 8, bFull = bars + 16, bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS,
                 bDp = bS + 8, bP = bDp + 8, bDs = bP + 8, bEnd = bDs + 8, bLse = bEnd + 16, bDelta = bLse + 8;
  uint32_t* const tmem_ptr = misc + 64;
  uint32_t* const stop_flag = misc + 65;
  float* const s_lse = reinterpret_cast<float*>(misc + 72);  // lse log2(e) of a tile's queries
  float* const s_delta = s_lse + kRows;

  if (warp == 8 && lane == 0) {
    *stop_flag = 0;
    bar_init(bKV, 1);
    bar_init(bKVfree, 1);
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 1);
    }
    bar_init(bS, 1);
    bar_init(bDp, 1);
    bar_init(bP, 8);
    bar_init(bDs, 8);
    bar_init(bEnd, 1);
    bar_init(bEnd + 8, 1);
    bar_init(bLse, 1);
    bar_init(bDelta, 1);
    bar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  if (blockIdx.x == 0 && warp == 0) check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(*tmem_ptr), tS = tm, tDp = tm + 128, tDv = tm + 256, tDk = tm + 384;
  const Stop stop{stop_flag, a.hdr};
  bool ok = true;
  asm volatile("griddepcontrol.launch_dependents;");  // the last kernel's blocks come beside this one's
  if (tid == 0) a.cut[blockIdx.x].parts = 0;

  // this block's turns [p0, p1), and its walk over them: key tile by key tile, pairs [u0, u1) of each
  KeyTile w;
  const int64_t all = find_turn(a, -1, &w), blocks = sharers(all, gridDim.x);
  const int64_t p0 = blockIdx.x < blocks ? share(all, blocks, blockIdx.x) : 0;
  const int64_t p1 = blockIdx.x < blocks ? share(all, blocks, blockIdx.x + 1) : 0;
  if (p0 < p1) find_turn(a, p0, &w);
  int u0 = 0, u1 = 0;
  bool begun = false;
  // the next tile with pairs (any: of those without, too)
  const auto step = [&](bool any) {
    for (;;) {
      if (begun) {
        if (w.last() >= p1) return false;
        next_tile(a, &w);
      } else if (p0 >= p1) {
        return false;
      }
      begun = true;
      const int64_t pairs = w.first + kEnds;  // from here on
      u0 = (int)uniform(pairs < p0 ? (uint32_t)(p0 - pairs) : 0u);
      u1 = (int)uniform(w.last() <= p1 ? (uint32_t)w.n : pairs < p1 ? (uint32_t)(p1 - pairs) : 0u);
      if (w.n > 0 ? u0 < u1 : any) return true;
    }
  };
  const auto more = [&](bool any) { return __any_sync(0xffffffffu, step(any)); };
  const auto full = [&](uint32_t c) { return warp_wait(bFull + 8 * (c % NS), (c / NS) & 1, stop); };

  if (warp == 8) {
    // ---- copies: keys and values of a tile, then queries (qd even) and output gradients
    uint32_t qd = 0, seen = 0;
    while (ok && more(false)) {
      if (lane == 0) {
        const int b = a.cu_q ? 0 : w.seq;
        const auto load = [&](int u) {
          const uint32_t sl = qd % NS;
          if (qd >= NS && !bar_wait(bEmpty + 8 * sl, (qd / NS - 1) & 1, stop)) return false;
          bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            copy_in_4d(sR + sl * P::kTileBytes + c * kHalf, u & 1 ? &a.dout : &a.q, bFull + 8 * sl, 64 * c,
                       w.hk * a.G + u / 2 / w.per, (int)(w.g.qbeg + (int64_t)(u / 2 % w.per) * kRows), b);
          ++qd;
          return true;
        };
        // the first queries go ahead: their slots are free before the last keys are
        ok = load(2 * u0) && load(2 * u0 + 1) && (seen == 0 || bar_wait(bKVfree, (seen - 1) & 1, stop));
        if (ok) {
          bar_expect(bKV, 2 * P::kTileBytes);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c) {
            copy_in_4d(sK + c * kHalf, &a.k, bKV, 64 * c, w.hk, (int)(w.g.kbeg + w.g.t0), b);
            copy_in_4d(sV + c * kHalf, &a.v, bKV, 64 * c, w.hk, (int)(w.g.kbeg + w.g.t0), b);
          }
        }
        for (int u = 2 * u0 + 2; ok && u < 2 * u1; ++u) ok = load(u);
      }
      ++seen;
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp == 9 || warp == 10) {
    // ---- products: dv += P do and S of the next tile of queries (warp 9), dk += dS q and dP
    // of the next (warp 10)
    const int x = warp - 9;
    constexpr uint32_t dS = product_desc(128, 128, false, false);
    const uint32_t dO = product_desc(128, 16 * steps, false, true);
    const uint32_t first = x ? tDp : tS, second = x ? tDk : tDv, own = kmajor(x ? sV : sK);
    const uint32_t bFirst = x ? bDp : bS, bSecond = x ? bDs : bP;
    uint32_t t = 0, seen = 0;
    while (ok && more(false)) {
      const int n = u1 - u0;
      const bool two = x == 1 && uniform(two_parts(w.g)) != 0;
      if (!(ok = warp_wait(bKV, seen & 1, stop))) break;
      const auto scores = [&](uint32_t c) {
        if (!full(2 * c + x)) return false;
        const uint32_t rows = uniform(kmajor(sR) + ((2 * c + x) % NS) * (P::kTileBytes >> 4));
        if (elect()) {
          issue_kk<DP>(first, own, rows, dS, steps);
          commit1(bFirst);
        }
        __syncwarp();
        return true;
      };
      if (!(ok = scores(t))) break;
      for (int u = 0; u < n; ++u, ++t) {
        // dv takes the output gradients, dk the queries
        const uint32_t rows = uniform(mnmajor(sR, kHalf) + ((2 * t + 1 - x) % NS) * (P::kTileBytes >> 4));
        if (!(ok = full(2 * t + 1 - x))) break;
        if (!(ok = warp_wait(bSecond, t & 1, stop))) break;
        fence_after();
        if (elect()) {
          issue_tn64(second, first, rows, dO, u > 0);
          issue_tn64(second, first + 64, rows + (64 * kPitch >> 4), dO, true);
          if (two) {
            issue_tn64(second, first + 32, rows, dO, true);
            issue_tn64(second, first + 96, rows + (64 * kPitch >> 4), dO, true);
          }
          if (u + 1 == n) commit1(bEnd + 8 * x);
        }
        __syncwarp();
        if (u + 1 < n && !(ok = scores(t + 1))) break;
      }
      ++seen;
    }
  } else if (warp == 11) {
    // ---- row statistics: lse of the next tile of queries as soon as every warp has P, delta
    // once every warp has dS; loaded a tile ahead
    asm volatile("griddepcontrol.wait;" ::: "memory");  // for the queries' kernel, which may change delta
    uint32_t t = 0;
    float l[4], d[4];
    const auto load = [&](int u) {
      const int h = w.hk * a.G + u / w.per;
      const int64_t t0 = (int64_t)(u % w.per) * kRows;
      const int64_t at = ((int64_t)(a.cu_q ? 0 : w.seq) * a.Hq + h) * a.Tq + w.g.qbeg + t0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = lane + 32 * i;
        const bool on = t0 + r < w.g.nq;
        l[i] = on ? a.lse[at + r] * 1.44269504088896341f : INFINITY;  // past the sequence: p = 0
        d[i] = on ? a.delta[at + r] : 0.f;
      }
    };
    while (ok && more(false)) {
      load(u0);
      for (int u = u0; u < u1; ++u, ++t) {
        if (t > 0 && !(ok = warp_wait(bP, (t - 1) & 1, stop))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) s_lse[lane + 32 * i] = l[i];
        __syncwarp();
        if (lane == 0) bar_arrive(bLse);
        if (t > 0 && !(ok = warp_wait(bDs, (t - 1) & 1, stop))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) s_delta[lane + 32 * i] = d[i];
        __syncwarp();
        if (lane == 0) bar_arrive(bDelta);
        if (u + 1 < u1) load(u + 1);
      }
    }
  } else {
    // ---- P and dS: key r of the tile in lane r, 64 query columns a warpgroup
    const int x = warp / 4, r = tid - 128 * x;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    uint32_t t = 0, seen = 0;
    while (ok && more(true)) {
      const int n = w.n > 0 ? u1 - u0 : 0;
      const bool two = two_parts(w.g);
      for (int u = 0; u < n; ++u, ++t) {
        const int64_t left = w.g.nq - (int64_t)((u0 + u) % w.per) * kRows;
        const int here = left < kRows ? (int)left : kRows;  // queries
        if (!(ok = warp_wait(bLse, t & 1, stop))) break;
        if (!(ok = warp_wait(bS, t & 1, stop))) break;
        fence_after();
        uint32_t s[2][32];
        tmem_ld32(tS + lanes + 64 * x, s[0]);
        tmem_ld32(tS + lanes + 64 * x + 32, s[1]);
        // the last tile's dv is done: its output gradients' slot is free
        if (tid == 0 && u > 0) bar_arrive(bEmpty + 8 * ((2 * t - 1) % NS));
        __syncwarp();
        ld_wait();
        const float2 sl2 = make_float2(a.sl2, a.sl2);
        const bool whole = here == kRows;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 from = *reinterpret_cast<const float4*>(s_lse + 64 * x + 32 * c + j);
            const float2 y = fma2(pair_of(s[c] + j), sl2, make_float2(-from.x, -from.y));
            const float2 z = fma2(pair_of(s[c] + j + 2), sl2, make_float2(-from.z, -from.w));
            s[c][j] = __float_as_uint(fast_exp2(y.x));
            s[c][j + 1] = __float_as_uint(fast_exp2(y.y));
            s[c][j + 2] = __float_as_uint(fast_exp2(z.x));
            s[c][j + 3] = __float_as_uint(fast_exp2(z.y));
          }
        if (!whole) {  // queries past the sequence may be anything
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (64 * x + 32 * c + j >= here) s[c][j] = 0u;
        }
        {
          // P and, below, dS go to the products as bf16, the type that the tensor cores take
          // next to bf16 operands: off by 2^-8 of themselves at most (dS as two parts, by
          // 2^-16). dS is formed from the P of 32 bits, and all sums are of 32 bits.
          uint32_t o[32];
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[16 * c + j] = pack_bf16(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1]));
          tmem_st32(tS + lanes + 64 * x, o);
        }
        if (!whole && a.cu_q) {  // rows of the next sequence
          if (!(ok = full(2 * t + 1))) break;
          clear_rows<DP>(sR + ((2 * t + 1) % NS) * P::kTileBytes, here, tid);
        }
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bP);
        __syncwarp();
        if (!(ok = warp_wait(bDelta, t & 1, stop))) break;
        if (!(ok = warp_wait(bDp, t & 1, stop))) break;
        fence_after();
        uint32_t d[2][32];
        tmem_ld32(tDp + lanes + 64 * x, d[0]);
        tmem_ld32(tDp + lanes + 64 * x + 32, d[1]);
        // the last tile's dk is done: its queries' slot is free
        if (tid == 0) {
          if (u > 0) bar_arrive(bEmpty + 8 * ((2 * t - 2) % NS));
          if (u + 1 == n) bar_arrive(bKVfree);
        }
        __syncwarp();
        ld_wait();
        uint32_t o[32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 less = *reinterpret_cast<const float4*>(s_delta + 64 * x + 32 * c + j);
            const float2 y = mul2(pair_of(s[c] + j), add2(pair_of(d[c] + j), make_float2(-less.x, -less.y)));
            const float2 z = mul2(pair_of(s[c] + j + 2), add2(pair_of(d[c] + j + 2), make_float2(-less.z, -less.w)));
            o[16 * c + j / 2] = pack_bf16(y.x, y.y);
            o[16 * c + j / 2 + 1] = pack_bf16(z.x, z.y);
            s[c][j] = __float_as_uint(y.x), s[c][j + 1] = __float_as_uint(y.y);
            s[c][j + 2] = __float_as_uint(z.x), s[c][j + 3] = __float_as_uint(z.y);
          }
        const auto cut_off = [&]() {  // what lies past the queries may be anything
          if (whole) return;
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int c = 64 * x + 2 * j;
            o[j] &= c + 1 < here ? 0xffffffffu : c < here ? 0xffffu : 0u;
          }
        };
        cut_off();
        tmem_st32(tDp + lanes + 64 * x, o);
        if (two) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            o[j] = rest_bf16(o[j], __uint_as_float(s[j / 16][2 * j % 32]), __uint_as_float(s[j / 16][2 * j % 32 + 1]));
          cut_off();
          tmem_st32(tDp + lanes + 64 * x + 32, o);
        }
        if (!whole && a.cu_q) clear_rows<DP>(sR + (2 * t % NS) * P::kTileBytes, here, tid);
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bDs);
        __syncwarp();
      }
      if (!ok) break;
      if (n > 0) {
        if (!(ok = warp_wait(bEnd, seen & 1, stop) && warp_wait(bEnd + 8, seen & 1, stop))) break;
        ++seen;
        fence_after();
        if (tid == 0) {  // the last tile's slots
          bar_arrive(bEmpty + 8 * ((2 * t - 1) % NS));
          bar_arrive(bEmpty + 8 * ((2 * t - 2) % NS));
        }
        __syncwarp();
      }
      // ---- warpgroup 0 writes dv, warpgroup 1 dk
      const uint32_t sum = (x == 0 ? tDv : tDk) + lanes;
      const int64_t key = w.g.t0 + r;
      const int b = a.cu_q ? 0 : w.seq;
      __nv_bfloat16* const out = x == 0 ? a.dvp + b * a.dv_sb + (w.g.kbeg + key) * a.dv_st + w.hk * a.dv_sh
                                        : a.dkp + b * a.dk_sb + (w.g.kbeg + key) * a.dk_st + w.hk * a.dk_sh;
      const bool cut = n > 0 && n < w.n, live = key < w.g.nk;
      if (cut && u0 == 0 && tid == 0) {
        int e = blockIdx.x;  // the block with its last pair
        while (share(all, blocks, e + 1) < w.last()) ++e;
        const int64_t left = w.g.nk - w.g.t0, rows = (a.cu_q ? w.g.nk : a.Tk) - w.g.t0;
        a.cut[blockIdx.x] = Cut{e - (int)blockIdx.x + 1, b, w.hk, (int)(left < kRows ? left : kRows), w.g.kbeg + w.g.t0,
                                rows < kRows ? rows : kRows};
      }
      if (cut) {
        // the parts of a tile that began in an earlier block's share go to the first place; four
        // columns of neighbouring rows lie side by side, as the threads of a warp have them (a row
        // in one piece: 6 us a tile)
        float* const to = a.part + (((int64_t)blockIdx.x * 2 + (u0 > 0 ? 0 : 1)) * 2 + x) * kRows * a.D + 4 * r;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(sum + 32 * c, o);
          ld_wait();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            if (32 * c + j < a.D)
              *reinterpret_cast<uint4*>(to + (32 * c + j) * kRows) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        }
      } else {
        if (n > 0) write_row<DP>(sum, x == 0 ? 1.f : a.scale, live, a.wide_kv, out, a.D);
        // no query sees these keys, or they are padding
        zero_row(n > 0 ? !live && !a.cu_q && key < a.Tk : live || (!a.cu_q && key < a.Tk), out, a.D);
      }
      fence_before();
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

// Adds the parts of the tile that block blockIdx.x's share begins and does not end, in
// order: eight columns of a row a thread, neighbouring rows in neighbouring threads.
__global__ void __launch_bounds__(256) cross_parts_kernel(const __grid_constant__ BwdArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the keys' kernel to end
  const Cut w = a.cut[blockIdx.x];
  const int i = blockIdx.y * 256 + threadIdx.x, r = i % kRows, x = i / kRows % 2, c = i / kRows / 2 * 8;
  if (w.parts == 0 || c >= a.D || r >= w.rows) return;
  float4 s[2];
  s[0] = s[1] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < w.live) {
    // the first part is its block's last place, the others their blocks' first
    const int64_t size = (int64_t)2 * kRows * a.D, at = (int64_t)x * kRows * a.D + c * kRows + 4 * r;
#pragma unroll 4
    for (int k = 0; k < w.parts; ++k) {
      const float* const p = a.part + (2 * ((int64_t)blockIdx.x + k) + (k == 0 ? 1 : 0)) * size + at;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 e = *reinterpret_cast<const float4*>(p + 4 * j * kRows);
        s[j].x += e.x, s[j].y += e.y, s[j].z += e.z, s[j].w += e.w;
      }
    }
  }
  const float f = x == 0 ? 1.f : a.scale;
  __nv_bfloat16* const out = x == 0 ? a.dvp + w.b * a.dv_sb + (w.key + r) * a.dv_st + w.hk * a.dv_sh
                                    : a.dkp + w.b * a.dk_sb + (w.key + r) * a.dk_st + w.hk * a.dk_sh;
  *reinterpret_cast<uint4*>(out + c) = make_uint4(pack_bf16(s[0].x * f, s[0].y * f), pack_bf16(s[0].z * f, s[0].w * f),
                                                  pack_bf16(s[1].x * f, s[1].y * f), pack_bf16(s[1].z * f, s[1].w * f));
}

template <int DP>
cudaError_t launch_bwd(const BwdArgs& t, unsigned blocks, cudaStream_t s) {
  using P = Plan<DP>;
  static_assert(P::kSmem <= 232448, "fits a block's shared memory");
  cudaError_t e = cudaFuncSetAttribute(cross_dkv_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cross_dq_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_early(cross_dq_kernel<DP>, dim3((unsigned)(t.items < kBlocks ? t.items : kBlocks)), kThreads, P::kSmem, s, t);
  if (e == cudaSuccess) e = launch_early(cross_dkv_kernel<DP>, dim3(blocks), kThreads, P::kSmem, s, t);
  if (e == cudaSuccess && blocks > 1)
    e = launch_early(cross_parts_kernel, dim3(blocks, (2 * kRows * t.D / 8 + 255) / 256), 256, 0, s, t);
  return e;
}

// Blocks of the keys' kernel: no more than can have two pairs each.
int64_t key_blocks(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t n_seqs) {
  const double q = (double)((Tq + kRows - 1) / kRows + n_seqs), k = (double)((Tk + kRows - 1) / kRows + n_seqs);
  const double most = (double)B * (double)Hq * q * k / 2. + 1.;
  return most < kBlocks ? (int64_t)most : kBlocks;
}

}  // namespace

size_t cross_tc_bwd_floats(int64_t B, int64_t Tq, int64_t Tk, int64_t Hq, int64_t D, int64_t n_seqs) {
  if (Tq < 1 || Tk < 1) return 0;
  return (size_t)key_blocks(B, Tq, Tk, Hq, n_seqs) * (4 * kRows * (size_t)D + sizeof(Cut) / 4);
}

cudaError_t launch_cross_tc_bwd(const CrossArgs& a, cudaStream_t s) {
  BwdArgs t;
  if (!encode_heads_map(&t.q, a.q, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.k, a.k, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.v, a.v, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.dout, a.dout, a.B, a.Tq, a.Hq, a.D, kRows))
    return cudaErrorInvalidValue;
  t.dqp = static_cast<__nv_bfloat16*>(a.dq.ptr);
  t.dq_sb = a.dq.stride_b, t.dq_st = a.dq.stride_t, t.dq_sh = a.dq.stride_h;
  t.dkp = static_cast<__nv_bfloat16*>(a.dk.ptr);
  t.dk_sb = a.dk.stride_b, t.dk_st = a.dk.stride_t, t.dk_sh = a.dk.stride_h;
  t.dvp = static_cast<__nv_bfloat16*>(a.dv.ptr);
  t.dv_sb = a.dv.stride_b, t.dv_st = a.dv.stride_t, t.dv_sh = a.dv.stride_h;
  t.lse = a.lse;
  t.delta = a.delta;
  const unsigned blocks = (unsigned)key_blocks(a.B, a.Tq, a.Tk, a.Hq, a.n_seqs);
  t.part = a.ws;
  t.cut = reinterpret_cast<Cut*>(a.ws + (size_t)blocks * 4 * kRows * a.D);
  t.lens = a.lens, t.cu_q = a.cu_q, t.cu_k = a.cu_k;
  t.hdr = a.hdr;
  t.B = a.B, t.Tq = a.Tq, t.Tk = a.Tk;
  t.n_seqs = a.n_seqs;
  t.order = orders(a.lens, a.cu_q, a.n_seqs, a.B);
  t.Hq = a.Hq, t.Hk = a.Hk, t.G = a.Hq / a.Hk, t.D = a.D;
  t.tiles = (a.Tq + kRows - 1) / kRows + (a.cu_q ? a.n_seqs : 0);
  t.items = t.tiles * a.B * a.Hq;
  t.wide = rows_on_32(a.dq, a.B, a.Tq, a.Hq, a.D);
  t.wide_kv = rows_on_32(a.dk, a.B, a.Tk, a.Hk, a.D) && rows_on_32(a.dv, a.B, a.Tk, a.Hk, a.D);
  t.sl2 = a.scale * 1.44269504088896341f;
  t.scale = a.scale;
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
  cross_delta_kernel<<<(unsigned)((d.rows + 63) / 64), 256, 0, s>>>(d);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return a.D <= 64 ? launch_bwd<64>(t, blocks, s) : launch_bwd<128>(t, blocks, s);
}

}  // namespace scan
