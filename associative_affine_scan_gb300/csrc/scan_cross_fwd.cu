// scan_cross_fwd.cu -- attention to another sequence, forward, on the tensor cores
// (bf16 operands).
//
// A block takes two tiles of 128 queries that read the same keys -- two heads that
// share a key head where their number is even, else 256 rows of one head -- and walks
// the tiles of 128 keys of their sequence in one pass with the reference m and sum l of
// each row's softmax (after Milakov and Gimelshein, "Online normalizer calculation for
// softmax"):
//   s = scale q k, p = 2^(s log2(e) - m), l = sum p, o = sum p v; at the end o / l.
// Two products of 128 x 128 x D a tile against 128 exponentials a row, so the two
// tiles take turns: while one's softmax runs, the tensor cores work on the other's
// products. Roles: a copy warp (a ring of key and value tiles), a product warp and four
// softmax warps a query tile, a row a thread. Tensor memory holds both tiles' scores
// and outputs (4 x 128 columns); p replaces its scores there as bf16 and is read from
// there by the second product.
// m is the first tile's maximum and is kept while the weights stay in range: their sum,
// which is formed anyway, tells. Only where it has grown by 2^16 is the tile worked
// again from its own maximum (128 comparisons a row less in all others; with them, and
// outputs rescaled from 2^8 on, the case below took 166 us).
// A product takes the tensor cores as long as its issue blocks the warp, and each wait
// and commit between products some 80 cycles more: so the two tiles' products are issued
// by two warps, in turn, each with its waits behind it when its turn comes. It comes
// while the other's last two products run (one warp for both: 183 us; turns at the very
// end: 158 us). Handing p over in two parts, and scores in two, cost more than they hid.
// Encoders are short: a block stays for several pairs of tiles, and no role waits for
// the others between them. The next pair's keys and queries are copied and its first
// scores formed while this one's outputs are written.
//
// 4 x 4096 queries, 1500 keys, 16 heads of 128: 156 us, 1.29 PFLOP/s; 4096 keys: 354 us,
// 1.55 PFLOP/s. Bound by the chain of a tile: 1000 cycles of products, 1340 of softmax
// (512 of them the special-function unit's) and 600 to 700 of handing over, against
// 2 x 1000 of tensor time for the pair; a pair's beginning and end cost another 5500.
#include <atomic>

#include "scan_cross_phases.h"
#include "scan_cross_tc.h"
#include "scan_tc.cuh"

namespace scan {
namespace {

using namespace tc;

constexpr int kRows = 128;
// Two softmax roles of four warps; copies, products of either query tile, an idle warp.
constexpr int kThreads = 12 * 32;
constexpr uint32_t kHalf = kRows * kPitch;
// A softmax thread holds the 128 scores of a row: its warpgroups take the registers that
// the third gives up. The shares are what the block is launched with, 168 a thread.
constexpr int kRegs = 168, kRegsSoftmax = 208, kRegsRest = 88;
static_assert(2 * kRegsSoftmax + kRegsRest == 3 * kRegs, "a larger sum would wait for ever");
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
}
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
}
// The sum of a tile's weights from which on a row's maximum is taken anew: they are held
// as multiples of what the maximum's weight is, in formats of 8 exponent bits, so that
// nothing is lost below that. A row's sum of 2^24 tiles stays below 2^40, so that values up to
// 2^80 (what the entry point allows) are far from fp32's largest number.
constexpr float kGrown = 65536.f;

struct FwdArgs {
  CUtensorMap q, k, v;
  __nv_bfloat16* op;
  int64_t o_sb, o_st, o_sh;
  float* lse;
  const int32_t *lens, *cu_q, *cu_k;
  WsHeader* hdr;
  int64_t B, Tq, Tk;
  int64_t tiles, items;  // pairs of query tiles of a (batch row, head or two), and of all
  int n_seqs, Hq, G;
  int order;      // the longest sequences first
  int two_heads;  // the two tiles are two heads' (else 256 rows of one)
  int D;
  int wide;  // rows of outputs are on 32 bytes
  float sl2;  // scale log2(e)
};

template <int DP>
struct Plan {
  static constexpr int kTileBytes = kRows * DP * 2;
  static constexpr int kSlots = fwd_slots(DP);
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024 + 1024;
};

// A pair of query tiles.
struct Item {
  CrossRows g;
  int b, h0, hk;
  int n;  // tiles of keys
};
// False: there is no such pair. A whole warp.
__device__ __forceinline__ bool item_at(const FwdArgs& a, const Order& order, int64_t i, Item* w) {
  const int units = a.two_heads ? a.Hq / 2 : a.Hq, rows = a.two_heads ? kRows : 2 * kRows;
  if (a.order) {
    int64_t unit, tile;
    int s;
    if (!order.find(i, units, &s, &unit, &tile)) return false;
    w->g = rows_of(a.lens, a.cu_q, a.cu_k, a.Tq, a.Tk, s, tile * rows);
    w->b = a.cu_q ? 0 : s;
    w->h0 = (int)unit * (a.two_heads ? 2 : 1);
    w->hk = w->h0 / a.G;
    w->n = (int)((w->g.nk + kRows - 1) / kRows);
    return true;
  }
  const int64_t unit = i / a.tiles, tile = i - unit * a.tiles;
  w->b = (int)(unit / units);
  w->h0 = (int)(unit % units) * (a.two_heads ? 2 : 1);
  w->hk = w->h0 / a.G;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, w->b, tile, rows, false, &w->g)) return false;
  w->n = (int)((w->g.nk + kRows - 1) / kRows);
  return true;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) cross_fwd_kernel(const __grid_constant__ FwdArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = (int)uniform(tid / 32), lane = tid % 32;
  const uint32_t sQ = base, sKV = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bQ = bars, bQfree = bars + 8, bFull = bars + 16, bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS,
                 bP = bS + 16, bO = bP + 16, bTurn = bO + 16;
  uint32_t* const tmem_ptr = misc + 96;
  uint32_t* const stop_flag = tmem_ptr + 1;
  Order& order = *reinterpret_cast<Order*>(misc + 100);

  if (warp == 8 && lane == 0) {
    *stop_flag = 0;
    bar_init(bQ, 1);
    bar_init(bQfree, 2);  // from both softmax roles
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 2);
    }
    for (int x = 0; x < 2; ++x) {
      bar_init(bS + 8 * x, 1);
      bar_init(bP + 8 * x, 4);
      bar_init(bO + 8 * x, 1);
      bar_init(bTurn + 8 * x, 1);
    }
    bar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  if (blockIdx.x == 0 && warp == 0) check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  if (a.order && warp == 10)
    order.make(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.two_heads ? kRows : 2 * kRows,
               a.two_heads ? a.Hq / 2 : a.Hq);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(*tmem_ptr);  // scores 0, scores 1, outputs 0, outputs 1
  const Stop stop{stop_flag, a.hdr};
  bool ok = true;
  Item w;

  if (warp >= 8) {
    give_registers();
    if (warp == 8) {
      // ---- copies: keys (kv even) and values of tile after tile through the ring
      uint32_t kv = 0, seen = 0;  // copies so far, pairs of query tiles so far
      for (int64_t r = 0; ok && item_of(r, a.order) < a.items; ++r) {
        if (!item_at(a, order, item_of(r, a.order), &w) || w.n == 0) continue;
        if (lane == 0) {
          const auto load = [&](int u) {
            const uint32_t sl = kv % NS;
            if (kv >= NS && !bar_wait_here(bEmpty + 8 * sl, (kv / NS - 1) & 1, stop)) return false;
            bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
            for (int c = 0; c < DP / 64; ++c)
              copy_in_4d(sKV + sl * P::kTileBytes + c * kHalf, u & 1 ? &a.v : &a.k, bFull + 8 * sl, 64 * c, w.hk,
                         (int)(w.g.kbeg + (int64_t)(u / 2) * kRows), w.b);
            ++kv;
            return true;
          };
          ok = load(0) && (seen == 0 || bar_wait_here(bQfree, (seen - 1) & 1, stop));
          if (ok) {
            bar_expect(bQ, 2 * P::kTileBytes);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int c = 0; c < DP / 64; ++c)
                copy_in_4d(sQ + x * P::kTileBytes + c * kHalf, &a.q, bQ, 64 * c, w.h0 + (a.two_heads ? x : 0),
                           (int)(w.g.qbeg + w.g.t0 + (a.two_heads ? 0 : x * kRows)), w.b);
          }
          for (int u = 1; ok && u < 2 * w.n; ++u) ok = load(u);
        }
        ++seen;
        ok = __all_sync(0xffffffffu, ok);
      }
    } else if (warp < 11) {
      // ---- products of query tile x: the outputs of a tile of keys, then the scores of the
      // next, which may be the next pair's first
      const int x = warp - 9;
      constexpr uint32_t dS = product_desc(128, 128, false, false);
      // what D leaves of the DP columns is neither multiplied nor summed
      const int steps = (a.D + 15) / 16;
      const uint32_t dO = product_desc(128, 16 * steps, false, true);
      const uint32_t p = tm + 128 * x, o = tm + 256 + 128 * x, q = kmajor(sQ) + x * (P::kTileBytes >> 4);
      uint32_t kv = 0, t = 0, seen = 1;  // copies used, tiles of keys so far, pairs so far
      int64_t round = 0;
      const auto next_item = [&]() {
        for (; item_of(round, a.order) < a.items; ++round)
          if (item_at(a, order, item_of(round, a.order), &w) && w.n > 0) break;
        const bool some = __any_sync(0xffffffffu, item_of(round, a.order) < a.items);
        ++round;
        return some;
      };
      const auto full = [&](uint32_t c) { return warp_wait_here(bFull + 8 * (c % NS), (c / NS) & 1, stop); };
      // scores from the keys at k; `turn`: the other tile's products may follow
      const auto scores = [&](uint32_t k, bool turn) {
        if (elect()) {
#pragma unroll
          for (int c = 0; c < DP / 16; ++c) {
            if (c >= steps) break;
            if (turn && c == (steps > 2 ? steps - 2 : 0)) bar_arrive(bTurn + 8 * (x ^ 1));
            const uint32_t step = (c / 4) * (kHalf >> 4) + (c % 4) * 2;
            mma_ss1(p, q + step, k + step, dS, c > 0);
          }
          commit1(bS + 8 * x);
        }
        __syncwarp();
      };
      bool more = next_item();
      int left = (int)uniform(w.n);
      bool add = false;
      if (more && (ok = warp_wait_here(bQ, 0, stop) && full(0))) scores(kmajor(sKV), false);

      while (ok && more) {
        const uint32_t v = uniform(mnmajor(sKV, kHalf) + ((kv + 1) % NS) * (P::kTileBytes >> 4));
        const bool last = left == 1, again = add;
        if (!(ok = full(kv + 1))) break;
        kv += 2;
        add = true;
        if (--left == 0) {
          more = next_item();
          left = (int)uniform(w.n);
          add = false;
          if (more && !(ok = warp_wait_here(bQ, seen & 1, stop))) break;
          ++seen;
        }
        if (more && !(ok = full(kv))) break;
        const uint32_t k = uniform(kmajor(sKV) + (kv % NS) * (P::kTileBytes >> 4));
        if (!(ok = warp_wait_here(bP + 8 * x, t & 1, stop))) break;
        if (x + t > 0 && !(ok = warp_wait_here(bTurn + 8 * x, (x ? t : t - 1) & 1, stop))) break;
        fence_after();
        if (elect()) {
#pragma unroll
          for (int c = 0; c < 8; ++c) mma_ts1(o, p + 8 * c, v + c * (2048 >> 4), dO, again || c > 0);
          if (last) commit1(bO + 8 * x);
          if (!more) bar_arrive(bTurn + 8 * (x ^ 1));
        }
        __syncwarp();
        if (more) scores(k, true);
        ++t;
      }

    }
  } else {
    take_registers();
    // ---- softmax: row r of tile x in lane r
    const int x = warp / 4, r = tid - 128 * x;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const uint32_t tS = tm + 128 * x + lanes, tO = tm + 256 + 128 * x + lanes;

    uint32_t t = 0, kv = 0, seen = 0;
    for (int64_t round = 0; ok && item_of(round, a.order) < a.items; ++round) {
      if (!item_at(a, order, item_of(round, a.order), &w)) continue;
      float m = 0.f, l = 0.f;
      for (int u = 0; u < w.n; ++u, ++t, kv += 2) {
        const int here = w.g.nk - (int64_t)u * kRows < kRows ? (int)(w.g.nk - (int64_t)u * kRows) : kRows;  // keys
        if (!(ok = warp_wait_here(bS + 8 * x, t & 1, stop))) break;
        fence_after();
        uint32_t s[4][32];
        tmem_ld32(tS, s[0]);
        tmem_ld32(tS + 32, s[1]);
        // these scores being there says that the products issued before them are done: the
        // keys' slot, the last tile's values' and at the end the queries' may be filled anew
        if (warp % 4 == 0 && lane == 0) {
          bar_arrive(bEmpty + 8 * (kv % NS));
          if (kv > 0) bar_arrive(bEmpty + 8 * ((kv - 1) % NS));
          if (u == w.n - 1) bar_arrive(bQfree);
        }
        __syncwarp();
        ld_wait();
        tmem_ld32(tS + 64, s[2]);
        tmem_ld32(tS + 96, s[3]);
        if (here < kRows) {
          ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= here) s[c][j] = 0xff800000u;
        }
        const auto top = [&]() {
          float y[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) y[z] = fmaxf(__uint_as_float(s[0][z]), __uint_as_float(s[0][z + 4]));
#pragma unroll
          for (int j = 8; j < 128; j += 8)
#pragma unroll
            for (int z = 0; z < 4; ++z)
              y[z] = max3(y[z], __uint_as_float(s[j / 32][j % 32 + z]), __uint_as_float(s[j / 32][j % 32 + z + 4]));
          return fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * a.sl2;
        };
        if (u == 0) {
          ld_wait();
          m = top();
          m = m == -INFINITY ? 0.f : m;
        }
        // p goes to the product as bf16, the type that the tensor cores take next to bf16
        // values: each weight is off by 2^-8 of itself at most, the output by about one
        // rounding of its own type (0.0023 of it in the 2-norm, 0.0017 for its own rounding
        // alone). The sum l is of p before that, in fp32.
        float tot;
#pragma unroll 1
        for (int round = 0;; ++round) {
          float2 sum[4] = {};
          const float2 f2 = make_float2(-m, -m), sl2 = make_float2(a.sl2, a.sl2);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c == 2) ld_wait();
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 z = fma2(pair_of(s[c] + j), sl2, f2);
              const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
              sum[j / 2 % 4] = add2(sum[j / 2 % 4], p);
              o[j / 2] = pack_bf16(p.x, p.y);
            }
            tmem_st16(tS + 16 * c, o);  // over columns that have been read
          }
          const float2 z = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          tot = z.x + z.y;
          const bool grown = !(tot <= kGrown);
          if (round > 0 || !__any_sync(0xffffffffu, grown)) break;
          // such rows once more from this tile's maximum, the sum and the outputs scaled to
          // it (the products into those are done: this tile's scores were issued after them)
          const float mn = grown ? fmaxf(m, top()) : m, f = m == mn ? 1.f : fast_exp2(m - mn);
          if (u > 0) {
#pragma unroll 1
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * c, o);
              ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(tO + 32 * c, o);
            }
          }
          l *= f;
          m = mn;
        }
        l += tot;
        if (here < kRows && (a.cu_q || a.lens)) {
          // value rows past the sequence may hold anything: both roles clear them before
          // their products may start
          const uint32_t vs = (kv + 1) % NS;
          if (!(ok = warp_wait_here(bFull + 8 * vs, ((kv + 1) / NS) & 1, stop))) break;
          const uint32_t v = sKV + vs * P::kTileBytes;
          const int past = kRows - here;
          for (int j = r; j < past * 8 * (DP / 64); j += 128)
            st_shared16(v + (j / 8 / past) * kHalf + (here + j / 8 % past) * kPitch + (j % 8) * 16, 0, 0, 0, 0);
          fence_async();
        }
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bP + 8 * x);
        __syncwarp();
      }
      if (!ok) break;
      // ---- o / l, straight to its rows
      if (w.n > 0) {
        if (!(ok = warp_wait_here(bO + 8 * x, seen & 1, stop))) break;
        fence_after();
        ++seen;
      }
      const bool some = l > 0.f;
      const float inv = some ? 1.f / l : l;  // l is 0, or NaN
      const int64_t row = w.g.t0 + (a.two_heads ? 0 : x * kRows) + r;
      const int h = w.h0 + (a.two_heads ? x : 0);
      const bool live = row < w.g.nq;
      __nv_bfloat16* const out = a.op + w.b * a.o_sb + (w.g.qbeg + row) * a.o_st + h * a.o_sh;
      if (w.n == 0) {
        if (live)
          for (int c = 0; c < a.D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
      } else {
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t o[32], v[16];
          tmem_ld32(tO + 32 * c, o);
          ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = pack_bf16(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
          if (live && a.wide) {
            if (32 * c < a.D) st_global32(out + 32 * c, v);
            if (32 * c + 16 < a.D) st_global32(out + 32 * c + 16, v + 8);
          } else if (live) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
              if (32 * c + 2 * j < a.D)
                *reinterpret_cast<uint4*>(out + 32 * c + 2 * j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
          }
        }
      }
      if (live)
        a.lse[((int64_t)w.b * a.Hq + h) * a.Tq + w.g.qbeg + row] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
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

// Whether the kernel is launched with the registers that its warpgroups' shares are of: the
// compiler's choice, of which the launch bounds are the upper limit. Asked once.
template <int DP>
cudaError_t shares_fit(bool* fit) {
  static std::atomic<int> regs{0};
  int n = regs.load(std::memory_order_relaxed);
  if (n == 0) {
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, cross_fwd_kernel<DP>);
    if (e != cudaSuccess) return e;
    regs.store(n = f.numRegs, std::memory_order_relaxed);
  }
  *fit = n == kRegs;
  return cudaSuccess;
}

template <int DP>
cudaError_t launch_fwd(const FwdArgs& t, unsigned grid, cudaStream_t s) {
  static_assert(Plan<DP>::kSmem <= 232448, "fits a block's shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(cross_fwd_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<DP>::kSmem);
  if (e != cudaSuccess) return e;
  cross_fwd_kernel<DP><<<grid, kThreads, Plan<DP>::kSmem, s>>>(t);
  return cudaGetLastError();
}

}  // namespace

// bf16 operands that tensor copies can address.
bool cross_tc_fits(const CrossArgs& a, scan_dtype dt, bool backward) {
  if (dt != SCAN_BF16 || a.Tq < 1 || a.Tk < 1 || a.Hq < 1) return false;
  const auto q = [&](const scan_view4& v) { return heads_map_fits(v, a.B, a.Tq, a.Hq); };
  const auto k = [&](const scan_view4& v) { return heads_map_fits(v, a.B, a.Tk, a.Hk); };
  if (!q(a.q) || !k(a.k) || !k(a.v) || !q(a.o)) return false;
  return !backward || (q(a.dout) && q(a.dq) && k(a.dk) && k(a.dv));
}

cudaError_t launch_cross_tc_fwd(const CrossArgs& a, cudaStream_t s) {
  bool fit;
  const cudaError_t e = a.D <= 64 ? shares_fit<64>(&fit) : shares_fit<128>(&fit);
  if (e != cudaSuccess) return e;
  if (!fit) return launch_cross_general_fwd(a, SCAN_BF16, s);  // built by a compiler that took other registers
  FwdArgs t;
  if (!encode_heads_map(&t.q, a.q, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.k, a.k, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.v, a.v, a.B, a.Tk, a.Hk, a.D, kRows))
    return cudaErrorInvalidValue;
  t.op = static_cast<__nv_bfloat16*>(a.o.ptr);
  t.o_sb = a.o.stride_b, t.o_st = a.o.stride_t, t.o_sh = a.o.stride_h;
  t.lse = a.lse;
  t.lens = a.lens, t.cu_q = a.cu_q, t.cu_k = a.cu_k;
  t.hdr = a.hdr;
  t.B = a.B, t.Tq = a.Tq, t.Tk = a.Tk;
  t.n_seqs = a.n_seqs;
  t.Hq = a.Hq;
  t.G = a.Hq / a.Hk;
  t.two_heads = t.G % 2 == 0;
  t.order = orders(a.lens, a.cu_q, a.n_seqs, a.B);
  t.D = a.D;
  t.wide = rows_on_32(a.o, a.B, a.Tq, a.Hq, a.D);
  t.sl2 = a.scale * 1.44269504088896341f;
  const int rows = t.two_heads ? kRows : 2 * kRows;
  t.tiles = (a.Tq + rows - 1) / rows + (a.cu_q ? a.n_seqs : 0);
  t.items = t.tiles * a.B * (t.two_heads ? a.Hq / 2 : a.Hq);
  const unsigned grid = (unsigned)(t.items < 152 ? t.items : 152);
  return a.D <= 64 ? launch_fwd<64>(t, grid, s) : launch_fwd<128>(t, grid, s);
}

}  // namespace scan
