// scan_window_fwd.cu -- sliding-window attention with first tokens that stay
// visible, forward, on the tensor cores (bf16 operands).
//
// A block takes two tiles of 128 queries that read the same keys: two heads that
// share a key head where their number is even, else 256 rows of one head. It
// walks the tiles of 128 keys that the queries see -- those of the first tokens,
// then those of the window -- in one pass with the running maximum m and sum l of
// each row's softmax (Milakov and Gimelshein, "Online normalizer calculation for
// softmax"):
//   s = scale q k, p = 2^(s log2(e) - m), l = sum p, o = sum p v; at the end o / l.
// Two products of 128 x 128 x D a tile (1024 tensor cycles at D = 128) against
// 128 exponentials a row, so the two tiles take turns: while one's softmax runs,
// the tensor cores work on the other's products. Roles: a copy warp (a ring of
// key and value tiles), a product warp, four softmax warps a query tile, a row a
// thread. Tensor memory holds both tiles' scores and outputs (4 x 128 columns); p
// replaces its scores there as bf16 and is read from there by the second product,
// which starts on the first 64 keys while the others' exponentials are still being
// taken. Scores are read twice, for the maximum and for the exponentials, which is
// cheaper than registers for 128 of them.
// The maximum that p is taken from follows the true one only when that has grown
// by more than 2^8: until then p stays below 2^8, which changes no rounding (bf16
// and fp32 have the same exponents), and the outputs need no rescaling.
//
// 16384 tokens, 16 query heads of 128 over 4 key heads, window 2048: 269 us, 0.96 PFLOP/s
// of seen pairs; 2 x 4096 tokens, window 1024: 91 us, 0.67 PFLOP/s. The tensor cores are
// busy for half of a block's cycles: scores, weights and outputs pass from role to role
// twice a tile, and tiles at the window's edges and of the first tokens are worked in
// whole. A second product warp, one a query tile, took 306 us for 266 at the time.
#include "scan_tc.cuh"
#include "scan_window_tc.h"

namespace scan {
namespace {

using namespace tc;

constexpr int kRows = 128;
constexpr int kThreads = 10 * 32;  // two softmax roles of four warps, copies, products
constexpr uint32_t kHalf = kRows * kPitch;

struct FwdArgs {
  CUtensorMap q, k, v, o;
  __nv_bfloat16* op;
  int64_t o_sb, o_st, o_sh;
  float* lse;
  const int32_t* cu;
  WsHeader* hdr;
  int64_t Tq, Tk, W, S;
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

// A column number of a tile, or one before or past all of them.
__device__ __forceinline__ int clamp_col(int64_t v) { return (int)(v < -1 ? -1 : v > 200 ? 200 : v); }

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) window_fwd_kernel(const __grid_constant__ FwdArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kSlots;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const uint32_t sQ = base, sKV = base + 2 * P::kTileBytes;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(gen + (2 + NS) * P::kTileBytes);
  const uint32_t bars = smem_addr(misc);
  const uint32_t bQ = bars, bFull = bars + 8, bEmpty = bFull + 8 * NS, bS = bEmpty + 8 * NS, bP = bS + 16,
                 bO = bP + 32, bOut = bO + 16;
  uint32_t* const tmem_ptr = misc + (8 + 16 * NS + 80) / 4;
  uint32_t* const stop_flag = tmem_ptr + 1;

  if (a.cu && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0)
    check_seqlens(a.cu, a.n_seqs, a.Tq, a.hdr);
  TileRows g;
  if (!tile_rows(a.cu, a.n_seqs, a.Tq, a.Tk, blockIdx.x, a.two_heads ? kRows : 2 * kRows, &g)) return;
  const int units = a.two_heads ? a.Hq / 2 : a.Hq;
  const int b = blockIdx.y / units;
  const int h0 = (blockIdx.y % units) * (a.two_heads ? 2 : 1), hk = h0 / a.G;
  // tile x: head hx, rows from tx; the key tiles it sees
  const auto head = [&](int x) { return a.two_heads ? h0 + x : h0; };
  const auto first = [&](int x) { return a.two_heads ? g.t0 : g.t0 + x * kRows; };
  KeyTiles kt[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int64_t p = g.off + first(x);
    const int64_t rows = g.nq - first(x) < kRows ? g.nq - first(x) : kRows;
    kt[x] = rows > 0 ? key_tiles(p, p + rows - 1, g.nk, a.W, a.S, kRows) : KeyTiles{0, 0, -1};
  }
  KeyTiles all = kt[0];
  if (kt[1].last > all.last) {  // rows further on: the union of both lists
    if (all.last < 0) all = kt[1];
    all.last = kt[1].last;
  }
  // The u-th of these tiles is tile() of the sequence. Query tile x sees it where u is
  // at most hi and below sk (first tokens) or at least lo. (32-bit numbers: the product
  // warp's own instructions are time that the tensor cores wait.)
  const int n = (int)all.count();
  const int n_sink = (int)all.sink, near = (int)all.near;
  const int sk = (int)((a.S < (int64_t)n * kRows ? a.S : (int64_t)n * kRows) + kRows - 1) / kRows;
  const int lo0 = n_sink + (int)(kt[0].near - all.near), lo1 = n_sink + (int)(kt[1].near - all.near);
  const int hi0 = kt[0].last < 0 ? -1 : n_sink + (int)(kt[0].last - all.near);
  const int hi1 = kt[1].last < 0 ? -1 : n_sink + (int)(kt[1].last - all.near);
  const auto tile = [&](int u) { return u < n_sink ? u : near + (u - n_sink); };
  const auto visits = [&](int x, int u) {
    return u <= (x ? hi1 : hi0) && (u < sk || u >= (x ? lo1 : lo0));
  };

  // tile u / 2 of the keys (u even) or values into its slot
  const auto load = [&](int u) {
    const int sl = u % NS, t = (int)(g.kbeg + (int64_t)tile(u / 2) * kRows);
    bar_expect(bFull + 8 * sl, P::kTileBytes);
#pragma unroll
    for (int i = 0; i < DP / 64; ++i)
      copy_in_4d(sKV + sl * P::kTileBytes + i * kHalf, u & 1 ? &a.v : &a.k, bFull + 8 * sl, 64 * i, hk, t, b);
  };
  // the copy warp sets the barriers up and starts the first copies while the others prepare
  if (warp == 8 && lane == 0) {
    *stop_flag = 0;
    bar_init(bQ, 1);
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 2);  // from both query tiles
    }
    for (int x = 0; x < 2; ++x) {
      bar_init(bS + 8 * x, 1);
      bar_init(bP + 16 * x, 4);
      bar_init(bP + 16 * x + 8, 4);
      bar_init(bO + 8 * x, 1);
      bar_init(bOut + 8 * x, 4);
    }
    bar_init_fence();
    if (n > 0) {
      bar_expect(bQ, 2 * P::kTileBytes);
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < DP / 64; ++i)
          copy_in_4d(sQ + x * P::kTileBytes + i * kHalf, &a.q, bQ, 64 * i, head(x), (int)(g.qbeg + first(x)), b);
      for (int u = 0; u < NS && u < 2 * n; ++u) load(u);
    }
  }
  __syncwarp();
  if (warp == 9) tmem_alloc(smem_addr(tmem_ptr), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *tmem_ptr;  // scores 0, scores 1, outputs 0, outputs 1
  const Stop stop{stop_flag, a.hdr};

  if (warp == 8) {
    // ---- copies
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
      int seen[2] = {0, 0};  // second products issued
      bool ok = warp_wait(bQ, 0, stop);
      const auto scores = [&](int x, int u) {
        mma_kk<DP, kHalf, kHalf>(lead, tm + 128 * x, kmajor(sQ) + x * (P::kTileBytes >> 4),
                                 kmajor(sKV) + (2 * u % NS) * (P::kTileBytes >> 4), dS, false);
        mma_commit(lead, bS + 8 * x);
      };
      ok = ok && warp_wait(bFull, 0, stop);
      if (ok) {
        for (int x = 0; x < 2; ++x)
          if (visits(x, 0)) scores(x, 0);
      }
      // What a softmax role hands over also says that the value tile, and the key tile
      // of the next scores, are there; and it is that role that gives slots back (its
      // scores arriving say that the products issued before them are done). Each wait
      // and each commit here would cost the tensor cores 100 to 200 cycles.
#pragma unroll 1
      for (int u = 0; ok && u < n; ++u) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const bool now = visits(x, u);
          if (now) {
            const uint32_t o = tm + 256 + 128 * x, p = tm + 128 * x;
            const uint32_t v = mnmajor(sKV, kHalf) + ((2 * u + 1) % NS) * (P::kTileBytes >> 4);
            if (!(ok = warp_wait(bP + 16 * x, seen[x] & 1, stop))) break;
            fence_after();
            mma_tn<64>(lead, o, p, v, dO, seen[x] > 0);
            if (!(ok = warp_wait(bP + 16 * x + 8, seen[x] & 1, stop))) break;
            fence_after();
            mma_tn<64>(lead, o, p + 32, v + (64 * kPitch >> 4), dO, true);
            if (u == (x ? hi1 : hi0)) mma_commit(lead, bO + 8 * x);
            ++seen[x];
          }
          if (u + 1 < n && visits(x, u + 1)) {
            if (!now && !(ok = warp_wait(bFull + 8 * ((2 * u + 2) % NS), ((2 * u + 2) / NS) & 1, stop))) break;
            scores(x, u + 1);
          }
        }
      }
    }
  } else {
    // ---- softmax: row r of tile x in lane r
    const int x = warp / 4, r = tid - 128 * x;
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const uint32_t tS = tm + 128 * x + lanes, tO = tm + 256 + 128 * x + lanes;
    const int64_t pos = g.off + first(x) + r;            // this row's position
    const int64_t wlo = g.off + first(x) + (warp % 4) * 32;  // the warp's first and last
    const int64_t whi = wlo + 31;
    float m = -INFINITY, l = 0.f;
    int k = 0;     // tiles seen
    int prev = 0, prev_u = 0;  // slot of the last one's values, and its number
    bool ok = true;
    for (int u = 0; u < n; ++u) {
      const int64_t j0 = (int64_t)tile(u) * kRows;
      const int ks = 2 * u % NS, vs = (2 * u + 1) % NS;
      if (!visits(x, u)) {  // nothing here for this tile; its slots' earlier uses are over
        if (warp % 4 == 0) {
          if (!(ok = warp_wait(bFull + 8 * ks, (2 * u / NS) & 1, stop))) break;
          if (!(ok = warp_wait(bFull + 8 * vs, ((2 * u + 1) / NS) & 1, stop))) break;
          if (lane == 0) {
            bar_arrive(bEmpty + 8 * ks);
            bar_arrive(bEmpty + 8 * vs);
          }
          __syncwarp();
        }
        continue;
      }
      const bool tail = a.cu && j0 + kRows > g.nk;  // the tile holds rows of the next sequence
      // Before the scores come: this tile's values and the next one's keys are there.
      // After a tile that was passed over, the slot of the values before it may be what
      // the next keys wait for: it is given back first, once the scores say that it can be.
      const bool passed = k > 0 && prev_u != u - 1;
      const auto next_keys = [&]() {
        return u + 1 >= n || warp_wait(bFull + 8 * ((2 * u + 2) % NS), ((2 * u + 2) / NS) & 1, stop);
      };
      if (warp % 4 == 0) {
        if (!(ok = warp_wait(bFull + 8 * vs, ((2 * u + 1) / NS) & 1, stop))) break;
        if (!passed && !(ok = next_keys())) break;
      }
      if (!(ok = warp_wait(bS + 8 * x, k & 1, stop))) break;
      fence_after();
      if (passed && warp % 4 == 0) {
        if (lane == 0) bar_arrive(bEmpty + 8 * prev);
        __syncwarp();
        if (!(ok = next_keys())) break;
      }
      const bool whole = j0 + kRows - 1 <= wlo && (whi - j0 < a.W || j0 + kRows <= a.S);
      if (!whole) {  // what this row does not see becomes -inf where it lies
        const int lo = clamp_col(pos - a.W + 1 - j0), hi = clamp_col(pos - j0), sk = clamp_col(a.S - j0);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          uint32_t s[32];
          tmem_ld32(tS + 32 * i, s);
          ld_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int j = 32 * i + c;
            if (!(j <= hi && (j >= lo || j < sk))) s[c] = 0xff800000u;
          }
          tmem_st32(tS + 32 * i, s);
        }
        st_wait();
      }
      float top;
      {
        uint32_t s[2][32];
        float y[4];
        tmem_ld32(tS, s[0]);
        ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the next columns are on their way while these are compared
          const uint32_t(&now)[32] = s[i & 1];
          if (i < 3) tmem_ld32(tS + 32 * (i + 1), s[(i + 1) & 1]);
#pragma unroll
          for (int c = 0; c < 32; c += 8)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float v = fmaxf(__uint_as_float(now[c + z]), __uint_as_float(now[c + z + 4]));
              y[z] = i == 0 && c == 0 ? v : fmaxf(y[z], v);
            }
          if (i < 3) ld_wait();
        }
        top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])) * a.sl2;
      }
      const bool grow = top > m + 8.f;  // from -inf: always, once a key is seen
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? top : m;
        const float f = m == mn ? 1.f : fast_exp2(m - mn);
        if (k > 0) {
          // (the products into it are done: this tile's scores were issued after them)
#pragma unroll 1
          for (int i = 0; i < DP / 32; ++i) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * i, o);
            ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
            tmem_st32(tO + 32 * i, o);
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
      {
        uint32_t s[2][32];
        tmem_ld32(tS, s[0]);
        ld_wait();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t(&now)[32] = s[i & 1];
          if (i < 3) tmem_ld32(tS + 32 * (i + 1), s[(i + 1) & 1]);
          uint32_t o[16];
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 z = fma2(pair_of(now + c), sl2, f2);
            const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
            sum[c / 2 % 4] = add2(sum[c / 2 % 4], p);
            o[c / 2] = pack_bf16(p.x, p.y);
          }
          if (i < 3) ld_wait();
          tmem_st16(tS + 16 * i, o);  // over columns that have been read
          if (i == 1) {
            st_wait();
            fence_before();
            __syncwarp();
            if (lane == 0 && !tail) bar_arrive(bP + 16 * x);
            __syncwarp();
          }
        }
      }
      {
        const float2 z = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += z.x + z.y;
      }
      if (tail) {
        // value rows past the sequence belong to the next one: both roles clear
        // them before their product may start
        if (!(ok = warp_wait(bFull + 8 * vs, ((2 * u + 1) / NS) & 1, stop))) break;
        const int from_row = (int)(g.nk - j0), left = kRows - from_row;
        const uint32_t v = sKV + vs * P::kTileBytes;
        for (int i = r; i < left * 8 * (DP / 64); i += 128)
          st_shared16(v + (i / 8 / left) * kHalf + (from_row + i / 8 % left) * kPitch + (i % 8) * 16, 0, 0, 0, 0);
        fence_async();
        __syncwarp();
      }
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (tail) bar_arrive(bP + 16 * x);
        bar_arrive(bP + 16 * x + 8);
        if (warp % 4 == 0) {
          bar_arrive(bEmpty + 8 * ks);
          if (k > 0 && !passed) bar_arrive(bEmpty + 8 * prev);
        }
      }
      __syncwarp();
      prev = vs;
      prev_u = u;
      ++k;
    }
    // ---- o / l to shared memory (the queries' place: their products are done), then out
    if (ok && k > 0) ok = warp_wait(bO + 8 * x, 0, stop);
    if (__all_sync(0xffffffffu, ok)) {
      fence_after();
      const bool some = l > 0.f;
      const float inv = some ? 1.f / l : l;  // l is 0, or NaN
      const int64_t row = first(x) + r;
      const bool live = row < g.nq;
      const bool direct = (a.cu && first(x) + kRows > g.nq) || k == 0;
      const uint32_t so = sQ + x * P::kTileBytes;
      __nv_bfloat16* const out = a.op + b * a.o_sb + (g.qbeg + row) * a.o_st + head(x) * a.o_sh;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        uint32_t o[32];
        if (k > 0) {
          tmem_ld32(tO + 32 * i, o);
          ld_wait();
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
          uint32_t w[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            w[y] = pack_bf16(__uint_as_float(o[c + 2 * y]) * inv, __uint_as_float(o[c + 2 * y + 1]) * inv);
          const int col = 32 * i + c;
          if (direct) {
            if (live && col < a.D) *reinterpret_cast<uint4*>(out + col) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
            st_shared16(swizzled(so + (col / 64) * kHalf, r, col % 64 / 8), w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live)
        a.lse[((int64_t)b * a.Hq + head(x)) * a.Tq + g.qbeg + row] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
      if (!direct) {
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(bOut + 8 * x);
        if (r == 0 && live && bar_wait(bOut + 8 * x, 0, stop)) {
#pragma unroll
          for (int i = 0; i < DP / 64; ++i)
            copy_out_4d(&a.o, so + i * kHalf, 64 * i, head(x), (int)(g.qbeg + first(x)), b);
          copy_out_commit();
          copy_out_done();
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

template <int DP>
cudaError_t launch_fwd(const FwdArgs& t, dim3 grid, cudaStream_t s) {
  static_assert(Plan<DP>::kSmem <= 232448, "fits a block's shared memory");
  const cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel<DP>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<DP>::kSmem);
  if (e != cudaSuccess) return e;
  window_fwd_kernel<DP><<<grid, kThreads, Plan<DP>::kSmem, s>>>(t);
  return cudaGetLastError();
}

}  // namespace

// bf16 operands that tensor copies can address.
bool window_tc_fits(const WinArgs& a, scan_dtype dt, bool backward) {
  if (dt != SCAN_BF16 || a.Tq < 1 || a.Tk < 1) return false;
  const auto q = [&](const scan_view4& v) { return heads_map_fits(v, a.B, a.Tq, a.Hq); };
  const auto k = [&](const scan_view4& v) { return heads_map_fits(v, a.B, a.Tk, a.Hk); };
  if (!q(a.q) || !k(a.k) || !k(a.v) || !q(a.o)) return false;
  return !backward || (q(a.dout) && q(a.dq) && k(a.dk) && k(a.dv));
}

cudaError_t launch_window_tc_fwd(const WinArgs& a, cudaStream_t s) {
  FwdArgs t;
  if (!encode_heads_map(&t.q, a.q, a.B, a.Tq, a.Hq, a.D, kRows) ||
      !encode_heads_map(&t.k, a.k, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.v, a.v, a.B, a.Tk, a.Hk, a.D, kRows) ||
      !encode_heads_map(&t.o, a.o, a.B, a.Tq, a.Hq, a.D, kRows))
    return cudaErrorInvalidValue;
  t.op = static_cast<__nv_bfloat16*>(a.o.ptr);
  t.o_sb = a.o.stride_b;
  t.o_st = a.o.stride_t;
  t.o_sh = a.o.stride_h;
  t.lse = a.lse;
  t.cu = a.cu;
  t.hdr = a.hdr;
  t.Tq = a.Tq;
  t.Tk = a.Tk;
  t.W = a.W;
  t.S = a.S;
  t.n_seqs = a.n_seqs;
  t.Hq = a.Hq;
  t.G = a.Hq / a.Hk;
  t.two_heads = t.G % 2 == 0;
  t.D = a.D;
  t.sl2 = a.scale * 1.44269504088896341f;
  const int rows = t.two_heads ? kRows : 2 * kRows;
  const int64_t tiles = (a.Tq + rows - 1) / rows + (a.cu ? a.n_seqs : 0);
  const dim3 grid((unsigned)tiles, (unsigned)(a.B * (t.two_heads ? a.Hq / 2 : a.Hq)));
  return a.D <= 64 ? launch_fwd<64>(t, grid, s) : launch_fwd<128>(t, grid, s);
}

}  // namespace scan
