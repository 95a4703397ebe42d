// scan_cross_fwd.cu -- attention to another sequence, forward, on the tensor cores
// (bf16 operands).
//
// A block takes two tiles of 128 queries that read the same keys -- two heads that
// share a key head where their number is even, else 256 rows of one head -- and walks
// the tiles of 128 keys of their sequence in one pass with the running maximum m and
// sum l of each row's softmax (Milakov and Gimelshein, "Online normalizer calculation
// for softmax"):
//   s = scale q k, p = 2^(s log2(e) - m), l = sum p, o = sum p v; at the end o / l.
// Two products of 128 x 128 x D a tile against 128 exponentials a row, so the two
// tiles take turns: while one's softmax runs, the tensor cores work on the other's
// products. Roles: a copy warp (a ring of key and value tiles), a product warp, four
// softmax warps a query tile, a row a thread. Tensor memory holds both tiles' scores
// and outputs (4 x 128 columns); p replaces its scores there as bf16 and is read from
// there by the second product, which starts on the first 64 keys while the others'
// exponentials are still being taken.
// Encoders are short: a block stays for several pairs of tiles, and no role waits for
// the others between them. The next pair's keys and queries are copied and its first
// scores formed while this one's outputs are written.
// The maximum that p is taken from follows the true one only when that has grown by
// more than 2^8: until then p stays below 2^8, which changes no rounding (bf16 and
// fp32 have the same exponents), and the outputs need no rescaling.
#include "scan_cross_tc.h"
#include "scan_tc.cuh"

namespace scan {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kThreads = 10 * 32;  // two softmax roles of four warps, copies, products
constexpr uint32_t kHalf = kRows * kPitch;

struct FwdArgs {
  CUtensorMap q, k, v;
  __nv_bfloat16* o;
  int64_t o_sb, o_st, o_sh;
  float* lse;
  const int32_t *lens, *cu_q, *cu_k;
  WsHeader* hdr;
  int64_t B, Tq, Tk;
  int64_t tiles, items;  // pairs of query tiles of a (batch row, head or two), and of all
  int n_seqs, Hq, G;
  int two_heads;  // the two tiles are two heads' (else 256 rows of one)
  int D;
  float sl2;  // scale log2(e)
};

template <int DP>
struct Plan {
  static constexpr int kTileBytes = kRows * DP * 2;
  static constexpr int kSlots = DP == 128 ? 5 : 8;
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024 + 512;
};

// A pair of query tiles.
struct Item {
  CrossRows g;
  int b, h0, hk;
  int n;  // tiles of keys
};
// False: there is no such pair. A whole warp.
__device__ __forceinline__ bool item_at(const FwdArgs& a, int64_t i, Item* w) {
  const int64_t unit = i / a.tiles, tile = i - unit * a.tiles;
  const int units = a.two_heads ? a.Hq / 2 : a.Hq;
  w->b = (int)(unit / units);
  w->h0 = (int)(unit % units) * (a.two_heads ? 2 : 1);
  w->hk = w->h0 / a.G;
  if (!cross_rows(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.Tq, a.Tk, w->b, tile, a.two_heads ? kRows : 2 * kRows, false, &w->g))
    return false;
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
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t sQ = base, sKV = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bQ = bars, bQfree = bars + 8, bFull = bars + 16, bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS,
                 bP = bS + 16, bO = bP + 32;
  uint32_t* const tmem_ptr = misc + 96;
  uint32_t* const stop_flag = tmem_ptr + 1;

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
      bar_init(bP + 16 * x, 4);
      bar_init(bP + 16 * x + 8, 4);
      bar_init(bO + 8 * x, 1);
    }
    bar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  if (blockIdx.x == 0 && warp == 0) check_cross(a.lens, a.cu_q, a.cu_k, a.n_seqs, a.B, a.Tq, a.Tk, a.hdr);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *tmem_ptr;  // scores 0, scores 1, outputs 0, outputs 1
  const Stop stop{stop_flag, a.hdr};
  bool ok = true;
  Item w;

  if (warp == 8) {
    // ---- copies: keys (kv even) and values of tile after tile through the ring
    uint32_t kv = 0, seen = 0;  // copies so far, pairs of query tiles so far
    for (int64_t i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
      if (!item_at(a, i, &w) || w.n == 0) continue;
      if (lane == 0) {
        const auto load = [&](int u) {
          const uint32_t sl = kv % NS;
          if (kv >= NS && !bar_wait(bEmpty + 8 * sl, (kv / NS - 1) & 1, stop)) return false;
          bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
          for (int c = 0; c < DP / 64; ++c)
            copy_in_4d(sKV + sl * P::kTileBytes + c * kHalf, u & 1 ? &a.v : &a.k, bFull + 8 * sl, 64 * c, w.hk,
                       (int)(w.g.kbeg + (int64_t)(u / 2) * kRows), w.b);
          ++kv;
          return true;
        };
        ok = load(0) && (seen == 0 || bar_wait(bQfree, (seen - 1) & 1, stop));
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
  } else if (warp == 9) {
    // ---- products, in the order scores and outputs of the two tiles by turns; the scores
    // of the next tile of keys, which may be the next pair's first, follow the outputs
    const bool lead = lane == 0;
    constexpr uint32_t dS = product_desc(128, 128, false, false);
    constexpr uint32_t dO = product_desc(128, DP, false, true);
    uint32_t kv = 0, t = 0, seen = 0;  // copies used, tiles of keys so far, pairs so far
    int64_t i = blockIdx.x;
    const auto next_item = [&]() {
      for (; i < a.items; i += gridDim.x)
        if (item_at(a, i, &w) && w.n > 0) break;
      const bool some = i < a.items;
      i += gridDim.x;
      return some;
    };
    const auto scores = [&](int x, uint32_t c) {
      mma_kk<DP, kHalf, kHalf>(lead, tm + 128 * x, kmajor(sQ) + x * (P::kTileBytes >> 4),
                               kmajor(sKV) + (c % NS) * (P::kTileBytes >> 4), dS, false);
      mma_commit(lead, bS + 8 * x);
    };
    bool more = next_item();
    int left = w.n, u = 0;
    if (more) {
      ok = warp_wait(bQ, 0, stop) && warp_wait(bFull, 0, stop);
      if (ok) {
        scores(0, 0);
        scores(1, 0);
      }
      ++seen;
    }
    while (ok && more) {
      const uint32_t v = mnmajor(sKV, kHalf) + ((kv + 1) % NS) * (P::kTileBytes >> 4);
      const bool add = u > 0, last = left == 1;
      const uint32_t full = (kv + 1) % NS, par = ((kv + 1) / NS) & 1;
      kv += 2;
      ++u;
      if (--left == 0) {
        more = next_item();
        left = w.n;
        u = 0;
      }
      if (!(ok = warp_wait(bFull + 8 * full, par, stop))) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t o = tm + 256 + 128 * x, p = tm + 128 * x;
        if (!(ok = warp_wait(bP + 16 * x, t & 1, stop))) break;
        fence_after();
        mma_tn<64>(lead, o, p, v, dO, add);
        if (!(ok = warp_wait(bP + 16 * x + 8, t & 1, stop))) break;
        fence_after();
        mma_tn<64>(lead, o, p + 32, v + (64 * kPitch >> 4), dO, true);
        if (last) mma_commit(lead, bO + 8 * x);
        if (more) {
          if (x == 0) {
            if (last && !(ok = warp_wait(bQ, seen & 1, stop))) break;
            if (!(ok = warp_wait(bFull + 8 * (kv % NS), (kv / NS) & 1, stop))) break;
          }
          scores(x, kv);
        }
      }
      if (last) ++seen;
      ++t;
    }
  } else {
    // ---- softmax: row r of tile x in lane r
    const int x = warp / 4, r = tid - 128 * x;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const uint32_t tS = tm + 128 * x + lanes, tO = tm + 256 + 128 * x + lanes;
    uint32_t t = 0, kv = 0, seen = 0;
    for (int64_t i = blockIdx.x; ok && i < a.items; i += gridDim.x) {
      if (!item_at(a, i, &w)) continue;
      float m = -INFINITY, l = 0.f;
      for (int u = 0; u < w.n; ++u, ++t, kv += 2) {
        const int here = w.g.nk - (int64_t)u * kRows < kRows ? (int)(w.g.nk - (int64_t)u * kRows) : kRows;  // keys
        if (!(ok = warp_wait(bS + 8 * x, t & 1, stop))) break;
        fence_after();
        // these scores being there says that the products issued before them are done: the
        // keys' slot, the last tile's values' and at the end the queries' may be filled anew
        if (warp % 4 == 0 && lane == 0) {
          bar_arrive(bEmpty + 8 * (kv % NS));
          if (kv > 0) bar_arrive(bEmpty + 8 * ((kv - 1) % NS));
          if (u == w.n - 1) bar_arrive(bQfree);
        }
        __syncwarp();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
        ld_wait();
        if (here < kRows) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= here) s[c][j] = 0xff800000u;
        }
        float y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) y[z] = fmaxf(__uint_as_float(s[0][z]), __uint_as_float(s[0][z + 4]));
#pragma unroll
        for (int j = 8; j < 128; j += 8)
#pragma unroll
          for (int z = 0; z < 4; ++z)
            y[z] = fmaxf(y[z], fmaxf(__uint_as_float(s[j / 32][j % 32 + z]), __uint_as_float(s[j / 32][j % 32 + z + 4])));
        const float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * a.sl2;
        const bool grow = top > m + 8.f;  // from -inf: always
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? top : m;
          const float f = m == mn ? 1.f : fast_exp2(m - mn);
          if (u > 0) {
            // (the products into it are done: this tile's scores were issued after them)
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
        const float from = m == -INFINITY ? 0.f : m;
        // p goes to the product as bf16, the type that the tensor cores take next to bf16
        // values: each weight is off by 2^-9 of itself at most, the output by about one
        // rounding of its own type. The sum l is of p before that, in fp32.
        float2 sum[4] = {};
        const float2 f2 = make_float2(-from, -from), sl2 = make_float2(a.sl2, a.sl2);
        const bool clear = here < kRows && (a.cu_q || a.lens);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 z = fma2(pair_of(s[c] + j), sl2, f2);
            const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
            sum[j / 2 % 4] = add2(sum[j / 2 % 4], p);
            o[j / 2] = pack_bf16(p.x, p.y);
          }
          tmem_st16(tS + 16 * c, o);  // over columns that have been read
          if (c == 1 && !clear) {
            st_wait();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bP + 16 * x);
            __syncwarp();
          }
        }
        {
          const float2 z = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l += z.x + z.y;
        }
        if (clear) {
          // value rows past the sequence may hold anything: both roles clear them before
          // their product may start
          const uint32_t vs = (kv + 1) % NS;
          if (!(ok = warp_wait(bFull + 8 * vs, ((kv + 1) / NS) & 1, stop))) break;
          const uint32_t v = sKV + vs * P::kTileBytes;
          const int past = kRows - here;
          for (int j = r; j < past * 8 * (DP / 64); j += 128)
            st_shared16(v + (j / 8 / past) * kHalf + (here + j / 8 % past) * kPitch + (j % 8) * 16, 0, 0, 0, 0);
          fence_async();
          __syncwarp();
        }
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if (clear) bar_arrive(bP + 16 * x);
          bar_arrive(bP + 16 * x + 8);
        }
        __syncwarp();
      }
      if (!ok) break;
      // ---- o / l, straight to its rows
      if (w.n > 0) {
        if (!(ok = warp_wait(bO + 8 * x, seen & 1, stop))) break;
        fence_after();
        ++seen;
      }
      const bool some = l > 0.f;
      const float inv = some ? 1.f / l : l;  // l is 0, or NaN
      const int64_t row = w.g.t0 + (a.two_heads ? 0 : x * kRows) + r;
      const int h = w.h0 + (a.two_heads ? x : 0);
      const bool live = row < w.g.nq;
      __nv_bfloat16* const out = a.o + w.b * a.o_sb + (w.g.qbeg + row) * a.o_st + h * a.o_sh;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        uint32_t o[32];
        if (w.n > 0) {
          tmem_ld32(tO + 32 * c, o);
          ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t v[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            v[z] = pack_bf16(__uint_as_float(o[j + 2 * z]) * inv, __uint_as_float(o[j + 2 * z + 1]) * inv);
          if (live && 32 * c + j < a.D) *reinterpret_cast<uint4*>(out + 32 * c + j) = make_uint4(v[0], v[1], v[2], v[3]);
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
  if (dt != SCAN_BF16 || a.Tq < 1 || a.Tk < 1) return false;
  const auto q = [&](const scan_view4& v) { return heads_map_fits(v, a.B, a.Tq, a.Hq); };
  const auto k = [&](const scan_view4& v) { return heads_map_fits(v, a.B, a.Tk, a.Hk); };
  if (!q(a.q) || !k(a.k) || !k(a.v) || !q(a.o)) return false;
  return !backward || (q(a.dout) && q(a.dq) && k(a.dk) && k(a.dv));
}

cudaError_t launch_cross_tc_fwd(const CrossArgs& a, cudaStream_t s) {
  FwdArgs t;
  if (!encode_heads_map(&t.q, a.q, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.k, a.k, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.v, a.v, a.B, a.Tk, a.Hk, a.D, kRows))
    return cudaErrorInvalidValue;
  t.o = static_cast<__nv_bfloat16*>(a.o.ptr);
  t.o_sb = a.o.stride_b, t.o_st = a.o.stride_t, t.o_sh = a.o.stride_h;
  t.lse = a.lse;
  t.lens = a.lens, t.cu_q = a.cu_q, t.cu_k = a.cu_k;
  t.hdr = a.hdr;
  t.B = a.B, t.Tq = a.Tq, t.Tk = a.Tk;
  t.n_seqs = a.n_seqs;
  t.Hq = a.Hq;
  t.G = a.Hq / a.Hk;
  t.two_heads = t.G % 2 == 0;
  t.D = a.D;
  t.sl2 = a.scale * 1.44269504088896341f;
  const int rows = t.two_heads ? kRows : 2 * kRows;
  t.tiles = (a.Tq + rows - 1) / rows + (a.cu_q ? a.n_seqs : 0);
  t.items = t.tiles * a.B * (t.two_heads ? a.Hq / 2 : a.Hq);
  const unsigned grid = (unsigned)(t.items < 152 ? t.items : 152);
  return a.D <= 64 ? launch_fwd<64>(t, grid, s) : launch_fwd<128>(t, grid, s);
}

}  // namespace scan
