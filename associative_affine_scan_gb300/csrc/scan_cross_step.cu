// scan_cross_step.cu -- attention of one query token a request over its encoder's
// cached keys and values (bf16 caches).
//
// Bound by DRAM: each cached row is read once for the query heads that share it. Caches
// differ in length, so the tiles of 64 keys of all (request, key head) pairs are dealt
// out in order, in equal shares, to one block an SM. A copy warp keeps a ring of six
// such tiles (32 KB each at D = 128) on its way ahead of the arithmetic, across the
// borders of requests. Two groups of four warps take the tiles by turns, 16 keys a warp:
// scores of up to 16 query heads by m16n8k16 products, the running maximum and sum of
// each row, and the weights, in two bf16 parts, by the values. A warp keeps its own sums
// until the request's last tile; then the warps' are added in order. A request that a share's
// end cuts leaves its parts in the workspace (at most two a block), which a second kernel adds
// in order.
//
// 64 requests over 800 to 4096 keys, 16 heads of 128 over 4: 60 us (5.4 TB/s) and 7 us; one
// request over 1500 keys, 16 heads: 10 us and 8 us, all latency. The ring holds 192 KB an SM
// on their way.
#include "scan_cross_phases.h"
#include "scan_cross_tc.h"
#include "scan_tc.cuh"

namespace scan {
namespace {

using namespace tc;

constexpr int kKeys = 64;  // of a tile
constexpr int kWarps = 8;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kBlocks = 152;  // one an SM
constexpr int kHeads = 16;    // query heads of a unit
constexpr uint32_t kPanel = kKeys * kPitch;

// What a cut leaves: which unit, and the maximum (times log2(e)), sum and output of each head.
struct Part {
  int64_t unit;   // -1: none
  int64_t goes_on;
  float m[kHeads], l[kHeads];
};

struct StepArgs {
  CUtensorMap k, v;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  int64_t q_sb, q_sh, o_sb, o_sh;
  const int32_t *lens, *slots;
  int64_t n_slots, Tk, B;
  int Hk, G, D;
  int rounds;   // units of 16 heads that a key head's heads make
  float sl2;
  WsHeader* hdr;
  Part* part;   // [blocks][2]: the first and the last unit of a share
  float* out;   // [blocks][2][16][D]
};

template <int DP>
struct Plan {
  static constexpr int kTileBytes = kKeys * DP * 2;  // of keys or values
  static constexpr int kStages = step_stages(DP);
  static_assert(kStages % 2 == 0, "a stage belongs to one group");
  static constexpr int kRow = DP + 8;                // floats: rows eight apart lie in different banks
  static constexpr int kFold = 4 * 8 * kRow * 4;     // sums of four warps, eight heads
  static constexpr int kSmem = kStages * 2 * kTileBytes + kFold + 1024 + 2048;
};

__device__ __forceinline__ int64_t slot_of(const StepArgs& a, int64_t b) {
  const int64_t s = a.slots ? (int64_t)a.slots[b] : b;
  return s < 0 || s >= a.n_slots ? -1 : s;
}
__device__ __forceinline__ int64_t keys_at(const StepArgs& a, int64_t slot) {
  return slot < 0 ? 0 : keys_of(a.lens, slot, a.Tk);
}
// Tiles of request b's units; one that has no keys counts as one (its output is zeros).
__device__ __forceinline__ int64_t tiles_of(int64_t keys) { return keys > 0 ? (keys + kKeys - 1) / kKeys : 1; }

// A place in the order: request, unit (key head and round) within it, tile.
struct Place {
  int64_t b;
  int unit;
  int64_t tile, slot, keys, tiles;
  __device__ void request(const StepArgs& a, int64_t r) {
    b = r;
    slot = slot_of(a, r);
    keys = keys_at(a, slot);
    tiles = tiles_of(keys);
  }
  __device__ void next_unit(const StepArgs& a, int units) {
    tile = 0;
    if (++unit == units) {
      unit = 0;
      if (b + 1 < a.B) request(a, b + 1);
    }
  }
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// The compute warps alone.
__device__ __forceinline__ void sync_compute() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) cross_step_kernel(const __grid_constant__ StepArgs a) {
  using P = Plan<DP>;
  constexpr int NS = P::kStages, KK = DP / 16, NN = DP / 8;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  float* const fold = reinterpret_cast<float*>(gen + NS * 2 * P::kTileBytes);
  uint8_t* const misc = gen + NS * 2 * P::kTileBytes + P::kFold;
  const uint32_t bFull = smem_addr(misc), bEmpty = bFull + 8 * NS;
  float* const s_m = reinterpret_cast<float*>(misc + 256);  // [8 warps][16]
  float* const s_l = s_m + kWarps * kHeads;
  float* const s_sum = s_l + kWarps * kHeads;  // [16]
  __shared__ int64_t s_scan[kThreads / 32], s_place[3];
  __shared__ uint32_t stop_flag, s_quit;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int units = a.Hk * a.rounds;

  asm volatile("griddepcontrol.launch_dependents;");  // the second kernel's blocks come beside this one's
  if (tid == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&a.k) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&a.v) : "memory");
    stop_flag = s_quit = 0;
    for (int i = 0; i < NS; ++i) {
      bar_init(bFull + 8 * i, 1);
      bar_init(bEmpty + 8 * i, 4);
    }
    bar_init_fence();
  }
  // ---- this block's share: the tiles of all requests are summed, a few requests a thread
  const int64_t each = (a.B + kThreads - 1) / kThreads, r0 = tid * each;
  int64_t mine = 0;
  for (int64_t r = r0; r < r0 + each && r < a.B; ++r) mine += tiles_of(keys_at(a, slot_of(a, r)));
  int64_t upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += o;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += s_scan[i];
    all += s_scan[i];
  }
  const int64_t total = all * units, blocks = total < (int64_t)gridDim.x ? total : (int64_t)gridDim.x;
  const auto first = [&](int64_t c) { return total / blocks * c + (total % blocks) * c / blocks; };
  const int64_t p0 = blockIdx.x < blocks ? first(blockIdx.x) : 0, p1 = blockIdx.x < blocks ? first(blockIdx.x + 1) : 0;
  if (p0 < p1 && mine > 0 && p0 >= (before + upto - mine) * units && p0 < (before + upto) * units) {
    int64_t p = p0 - (before + upto - mine) * units, r = r0;
    for (;; ++r) {
      const int64_t n = tiles_of(keys_at(a, slot_of(a, r)));
      if (p < n * units) {
        s_place[0] = r;
        s_place[1] = p / n;
        s_place[2] = p % n;
        break;
      }
      p -= n * units;
    }
  }
  __syncthreads();
  Part* const part = a.part + 2 * blockIdx.x;
  if (tid < 2) part[tid].unit = -1;
  if (p0 >= p1) return;
  const Stop stop{&stop_flag, a.hdr};
  Place w;
  w.request(a, s_place[0]);
  w.unit = (int)s_place[1];
  w.tile = s_place[2];
  bool ok = true;

  if (warp == kWarps) {
    // ---- copies: the keys and values of tile after tile
    if (lane == 0) {
      uint32_t n = 0;
      for (int64_t p = p0; ok && p < p1; ++p) {
        if (w.keys > 0) {
          const uint32_t sl = n % NS, to = base + sl * 2 * P::kTileBytes;
          if (n >= NS && !(ok = bar_wait(bEmpty + 8 * sl, (n / NS - 1) & 1, stop))) break;
          bar_expect(bFull + 8 * sl, 2 * P::kTileBytes);
          const int hk = w.unit / a.rounds;
#pragma unroll
          for (int c = 0; c < DP / 64; ++c) {
            copy_in_4d(to + c * kPanel, &a.k, bFull + 8 * sl, 64 * c, hk, (int)(w.tile * kKeys), (int)w.slot);
            copy_in_4d(to + P::kTileBytes + c * kPanel, &a.v, bFull + 8 * sl, 64 * c, hk, (int)(w.tile * kKeys), (int)w.slot);
          }
          ++n;
        }
        if (++w.tile == w.tiles) w.next_unit(a, units);
      }
    }
    __syncwarp();
    linger(stop);
    return;
  }

  const int grp = warp / 4, g = lane / 4, c = lane % 4;
  const int key0 = (warp % 4) * 16;  // this warp's keys of a tile
  uint32_t n = 0;                    // tiles so far, of both groups
  for (int64_t p = p0; ok && p < p1;) {
    // ---- a unit, or what the share has of it: tiles [w.tile, w.tile + count)
    const int64_t count = w.tiles - w.tile < p1 - p ? w.tiles - w.tile : p1 - p;
    const int h0 = (w.unit / a.rounds) * a.G + w.unit % a.rounds * kHeads;  // its first query head
    const int left = a.G - w.unit % a.rounds * kHeads, heads = left < kHeads ? left : kHeads;
    const __nv_bfloat16* const q = a.q + w.b * a.q_sb + h0 * a.q_sh;
    __nv_bfloat16* const o = a.o + w.b * a.o_sb + h0 * a.o_sh;
    if (w.keys == 0) {  // an idle request, or no keys
      for (int i = tid; i < heads * a.D; i += 32 * kWarps) o[i / a.D * a.o_sh + i % a.D] = __float2bfloat16_rn(0.f);
    } else {
      uint32_t qa[KK][4];
#pragma unroll
      for (int k = 0; k < KK; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = g + 8 * (i & 1), d = 16 * k + 2 * c + 8 * (i >> 1);
          qa[k][i] = h < heads && d < a.D ? *reinterpret_cast<const uint32_t*>(q + h * a.q_sh + d) : 0u;
        }
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, acc[NN][4];
#pragma unroll
      for (int i = 0; i < NN; ++i)
#pragma unroll
        for (int y = 0; y < 4; ++y) acc[i][y] = 0.f;
      for (int64_t t = 0; t < count; ++t, ++n) {
        if ((n & 1) != grp) continue;
        const uint32_t sl = n % NS, sk = base + sl * 2 * P::kTileBytes, sv = sk + P::kTileBytes;
        const int64_t here = w.keys - (w.tile + t) * kKeys - key0;  // this warp's keys, if below 16
        if (!(ok = warp_wait(bFull + 8 * sl, (n / NS) & 1, stop))) break;
        float s[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int y = 0; y < 4; ++y) s[x][y] = 0.f;
          const int row = key0 + 8 * x + lane % 8;
#pragma unroll
          for (int k = 0; k < KK; k += 2) {
            uint32_t b[4];
            const int piece = 2 * k + lane / 8;
            ldsm(b, swizzled(sk + (piece / 8) * kPanel, row, piece % 8));
            mma16816(s[x], qa[k], b[0], b[1]);
            mma16816(s[x], qa[k + 1], b[2], b[3]);
          }
        }
        // s[x][y], s[x][2 + y]: heads g and g + 8, key key0 + 8 x + 2 c + y
        if (here < 16) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (8 * x + 2 * c + y >= here) s[x][y] = s[x][2 + y] = -INFINITY;
        }
        float top[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2)) * a.sl2;
        }
        if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
          float keep[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], top[h]);
            keep[h] = m[h] == mn ? 1.f : fast_exp2(m[h] - mn);
            m[h] = mn;
            l[h] *= keep[h];
          }
#pragma unroll
          for (int i = 0; i < NN; ++i) {
            acc[i][0] *= keep[0];
            acc[i][1] *= keep[0];
            acc[i][2] *= keep[1];
            acc[i][3] *= keep[1];
          }
        }
        // (weights as the sum of two bf16 numbers, the type of the values they multiply: off by
        // 2^-16 of themselves at most. With one, off by 2^-8, the output's error in the 2-norm was
        // 0.0021 of it where its own rounding is 0.0017. l is the sum of the unrounded ones)
        uint32_t pa[4], rest[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float from = m[h] == -INFINITY ? 0.f : m[h];
          float e[2][2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              e[x][y] = fast_exp2(fmaf(s[x][2 * h + y], a.sl2, -from));
              l[h] += e[x][y];
            }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            pa[2 * x + h] = pack_bf16(e[x][0], e[x][1]);
            rest[2 * x + h] = rest_bf16(pa[2 * x + h], e[x][0], e[x][1]);
          }
        }
        uint32_t on[2] = {0xffffffffu, 0xffffffffu};  // which of the values' keys are there
        if (here < 16) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
            on[x] = 8 * x + 2 * c + 1 < here ? 0xffffffffu : 8 * x + 2 * c < here ? 0xffffu : 0u;
        }
        const int row = key0 + lane % 16;
#pragma unroll
        for (int i = 0; i < NN; i += 2) {
          uint32_t b[4];
          const int piece = i + lane / 16;
          ldsm_t(b, swizzled(sv + (piece / 8) * kPanel, row, piece % 8));
          b[0] &= on[0], b[1] &= on[1], b[2] &= on[0], b[3] &= on[1];
          mma16816(acc[i], pa, b[0], b[1]);
          mma16816(acc[i + 1], pa, b[2], b[3]);
          mma16816(acc[i], rest, b[0], b[1]);
          mma16816(acc[i + 1], rest, b[2], b[3]);
        }
        __syncwarp();
        if (lane == 0) bar_arrive(bEmpty + 8 * sl);
      }
      // ---- the warps' sums: scaled to their common maximum, then added in order
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        if (c == 0) s_m[warp * kHeads + 8 * h + g] = m[h], s_l[warp * kHeads + 8 * h + g] = l[h];
      }
      if (!ok && lane == 0) s_quit = 1;
      sync_compute();
      const bool quit = s_quit != 0;  // the warps leave together
      float f[2], top[2], sum[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = -INFINITY;
        for (int i = 0; i < kWarps; ++i) top[h] = fmaxf(top[h], s_m[i * kHeads + 8 * h + g]);
        const float from = top[h] == -INFINITY ? 0.f : top[h];
        f[h] = fast_exp2(m[h] - from);
        sum[h] = 0.f;
        for (int i = 0; i < kWarps; ++i)
          sum[h] = fmaf(s_l[i * kHeads + 8 * h + g], fast_exp2(s_m[i * kHeads + 8 * h + g] - from), sum[h]);
      }
      // eight heads at a time: the sums of warps 4 to 7 are added to those of warps 0 to 3,
      // then these four in order, by all threads
      const bool whole = count == w.tiles;
      const int place = w.tile > 0 ? 0 : 1;  // of a part: begun in an earlier share, or in this
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (8 * h >= heads) break;
        float* const at = fold + ((warp % 4) * 8 + g) * P::kRow + 2 * c;
#pragma unroll
        for (int i = 0; i < NN; ++i) acc[i][2 * h] *= f[h], acc[i][2 * h + 1] *= f[h];
        if (warp >= 4)
#pragma unroll
          for (int i = 0; i < NN; ++i) *reinterpret_cast<float2*>(at + 8 * i) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
        sync_compute();
        if (warp < 4)
#pragma unroll
          for (int i = 0; i < NN; ++i) {
            const float2 e = *reinterpret_cast<const float2*>(at + 8 * i);
            *reinterpret_cast<float2*>(at + 8 * i) = make_float2(acc[i][2 * h] + e.x, acc[i][2 * h + 1] + e.y);
          }
        if (warp == 0 && c == 0) {  // what the outputs are divided by, of each head
          s_sum[8 * h + g] = sum[h];
          if (!whole) part[place].m[8 * h + g] = top[h], part[place].l[8 * h + g] = sum[h];
        }
        sync_compute();
        if (!quit)
          for (int i = tid; i < 8 * (DP / 2); i += 32 * kWarps) {
            const int r = i / (DP / 2), d = 2 * (i % (DP / 2));
            if (8 * h + r >= heads || d >= a.D) continue;
            float2 e = *reinterpret_cast<const float2*>(fold + r * P::kRow + d);
#pragma unroll
            for (int k = 1; k < 4; ++k) {
              const float2 y = *reinterpret_cast<const float2*>(fold + (8 * k + r) * P::kRow + d);
              e.x += y.x, e.y += y.y;
            }
            if (whole) {
              const float inv = s_sum[8 * h + r] == 0.f ? 0.f : 1.f / s_sum[8 * h + r];
              *reinterpret_cast<uint32_t*>(o + (8 * h + r) * a.o_sh + d) = pack_bf16(e.x * inv, e.y * inv);
            } else {
              *reinterpret_cast<float2*>(a.out + ((2 * (int64_t)blockIdx.x + place) * kHeads + 8 * h + r) * a.D + d) = e;
            }
          }
        if (h == 0 && heads > 8) sync_compute();  // the place is free again
      }
      if (tid == 0 && !quit && !whole) {
        part[place].unit = w.b * units + w.unit;
        part[place].goes_on = w.tile + count < w.tiles;
      }
      ok = !quit;
    }
    p += count;
    w.tile += count;
    if (w.tile == w.tiles) w.next_unit(a, units);
  }
  linger(stop);
}

// Adds the parts of the unit whose first part is block blockIdx.x's last, in order.
__global__ void __launch_bounds__(256) cross_step_parts_kernel(const __grid_constant__ StepArgs a, int grid) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the first kernel's end
  const Part* const p = a.part + 2 * blockIdx.x + 1;
  const int64_t id = p->unit;
  if (id < 0) return;
  const int units = a.Hk * a.rounds;
  const int64_t b = id / units;
  const int unit = (int)(id - b * units);
  const int h0 = (unit / a.rounds) * a.G + unit % a.rounds * kHeads;
  const int left = a.G - unit % a.rounds * kHeads, heads = left < kHeads ? left : kHeads;
  int n = 0;  // blocks that share it, looked up 32 at a time
  for (int k0 = 1; n == 0; k0 += 32) {
    const int k = k0 + threadIdx.x % 32;
    const bool here = blockIdx.x + k < grid && a.part[2 * (blockIdx.x + k)].unit == id;
    const unsigned is = __ballot_sync(0xffffffffu, here);
    const unsigned ends = __ballot_sync(0xffffffffu, !here || a.part[2 * (blockIdx.x + k)].goes_on == 0);
    if (ends) {
      const int j = __ffs(ends) - 1;
      n = k0 + j + (is >> j & 1);
    }
  }
  for (int i = threadIdx.x; i < heads * a.D; i += 256) {
    const int h = i / a.D, d = i % a.D;
    float top = p->m[h];
#pragma unroll 8
    for (int k = 1; k < n; ++k) top = fmaxf(top, a.part[2 * (blockIdx.x + k)].m[h]);
    const float from = top == -INFINITY ? 0.f : top;
    float f = fast_exp2(p->m[h] - from);
    float sum = p->l[h] * f, e = a.out[((2 * (int64_t)blockIdx.x + 1) * kHeads + h) * a.D + d] * f;
#pragma unroll 8
    for (int k = 1; k < n; ++k) {
      const Part* const r = a.part + 2 * (blockIdx.x + k);
      f = fast_exp2(r->m[h] - from);
      sum = fmaf(r->l[h], f, sum);
      e = fmaf(a.out[(2 * (int64_t)(blockIdx.x + k) * kHeads + h) * a.D + d], f, e);
    }
    a.o[b * a.o_sb + (h0 + h) * a.o_sh + d] = __float2bfloat16_rn(sum == 0.f ? 0.f : e / sum);
  }
}

template <int DP>
cudaError_t launch_step(const StepArgs& t, unsigned grid, cudaStream_t s) {
  static_assert(Plan<DP>::kSmem <= 232448, "fits a block's shared memory");
  const cudaError_t e =
      cudaFuncSetAttribute(cross_step_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Plan<DP>::kSmem);
  if (e != cudaSuccess) return e;
  cross_step_kernel<DP><<<grid, kThreads, Plan<DP>::kSmem, s>>>(t);
  const cudaError_t made = cudaGetLastError();
  if (made != cudaSuccess) return made;
  return launch_early(cross_step_parts_kernel, dim3(grid), 256, 0, s, t, (int)grid);
}

// Blocks: no more than there can be tiles, two at least.
int64_t step_blocks(int64_t B, int64_t Tk, int64_t Hk, int64_t Hq) {
  const double rounds = Hk > 0 ? (double)((Hq / Hk + kHeads - 1) / kHeads) : 0.;
  const double most = (double)B * (double)Hk * rounds * (double)((Tk + kKeys - 1) / kKeys + 1);
  return most < kBlocks ? (int64_t)most : kBlocks;
}

}  // namespace

size_t cross_step_bytes(int64_t B, int64_t Tk, int64_t Hq, int64_t Hk, int64_t D) {
  return (size_t)step_blocks(B, Tk, Hk, Hq) * 2 * (sizeof(Part) + kHeads * (size_t)D * 4);
}

bool cross_step_fits(const CrossStepArgs& a, scan_dtype dt, int64_t B) {
  if (dt != SCAN_BF16 || a.Tk < 1 || a.n_slots < 1) return false;
  const auto even = [](const scan_view4& v) {  // heads of query and output are read by pairs
    return (uintptr_t)v.ptr % 4 == 0 && v.stride_b % 2 == 0 && v.stride_h % 2 == 0;
  };
  return heads_map_fits(a.k, a.n_slots, a.Tk, a.Hk) && heads_map_fits(a.v, a.n_slots, a.Tk, a.Hk) && even(a.q) &&
         even(a.o) && a.n_slots <= 0x7fffffffLL;
}

cudaError_t launch_cross_step(const CrossStepArgs& a, int64_t B, cudaStream_t s) {
  StepArgs t;
  if (!encode_heads_map(&t.k, a.k, a.n_slots, a.Tk, a.Hk, a.D, kKeys) ||
      !encode_heads_map(&t.v, a.v, a.n_slots, a.Tk, a.Hk, a.D, kKeys))
    return cudaErrorInvalidValue;
  t.q = static_cast<const __nv_bfloat16*>(a.q.ptr);
  t.o = static_cast<__nv_bfloat16*>(a.o.ptr);
  t.q_sb = a.q.stride_b, t.q_sh = a.q.stride_h, t.o_sb = a.o.stride_b, t.o_sh = a.o.stride_h;
  t.lens = a.lens, t.slots = a.slots;
  t.n_slots = a.n_slots, t.Tk = a.Tk, t.B = B;
  t.Hk = a.Hk, t.G = a.Hq / a.Hk, t.D = a.D;
  t.rounds = (t.G + kHeads - 1) / kHeads;
  t.sl2 = a.scale * 1.44269504088896341f;
  t.hdr = a.hdr;
  const int64_t blocks = step_blocks(B, a.Tk, a.Hk, a.Hq);
  t.part = static_cast<Part*>(a.ws);
  t.out = reinterpret_cast<float*>(t.part + 2 * blocks);
  return a.D <= 64 ? launch_step<64>(t, (unsigned)blocks, s) : launch_step<128>(t, (unsigned)blocks, s);
}

}  // namespace scan
