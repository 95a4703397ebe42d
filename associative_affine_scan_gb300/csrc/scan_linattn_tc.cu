// scan_linattn_tc.cu -- linear attention with a decay for each head, chunk by
// chunk on the tensor cores (bf16 operands).
//
// One pass over (x1, x2, x3) (see LinPass; forward: q, k, v), a chunk of 128
// steps at a time in the order of the recurrence. r counts a chunk's n steps in
// that order, e = 1 forward and 0 reversed, S (K x V) is the state before it:
//   out_r = scale ( lambda^(r + e) x1_r S + sum_{r' <= r} lambda^(r - r') (x1_r x2_r') x3_r' )
//   S    <- lambda^n S + sum_r' lambda^(n - e - r') x2_r' x3_r'^T
// Four products of 128^3 a chunk at K = V = 128 (the state's update twice, see
// below): 5 x 512 tensor cycles against the 5600 that one SM's share of DRAM
// needs for the chunk's 128 KB, so the kernel is bound by DRAM as long as copies,
// products and the conversions between them overlap. Roles of a block (one per
// SM), each working on its own part of the chain at any time:
//   copy warp     two to four chunks of x1, x2, x3 in flight
//   product warp  S1 = x1 x2^T, O = x1 S, S^T += x3'^T x2, O += P x3
//   weights       P = S1 * lambda^(r - r'), masked, to bf16 over S1
//   state         S^T to bf16 for the next chunk's x1 S, and S^T *= lambda^n
//   update        x3'^T = lambda^(n - e - r') x3^T as the sum of two bf16 parts (three
//                 where the state is an output), 32 steps at a time: the state's
//                 update is then exact to 2^-16 (2^-24), so that the state, fp32 in
//                 tensor memory, keeps that accuracy over any number of chunks
//   output        O *= lambda^(r + e) between the two products into it; O to bf16
// P, and the state as x1 reads it, are rounded once to bf16, the type that the tensor
// cores take next to bf16 operands: each term of an output is off by 2^-8 of itself at
// most, which is the size of the output's own rounding. Neither is carried on: the state
// itself and all sums stay in 32 bits.
// The state lies transposed (lanes are v): its bf16 copy is then written by rows
// into the operand layout, and the weighted operand of the update is one that the
// tensor cores read from tensor memory, which shared memory has no room for.
//
// Few (sequence, head) rows: each is cut into segments; the segments' own states
// are found first (x2 and x3 only), chained, and each segment then starts from
// the state before it. This reads x2 and x3 twice.
//
// Heads of 128 x 128, bf16. 16384 steps of 16 heads (one row): own states 31 us, chain
// 6 us, chunks 62 us (269 MB, 4.3 TB/s). 4 x 4096 steps of 16 heads: own states 19 us,
// chunks 61 us; backward, three passes at once, 213 us (805 MB, 3.8 TB/s). A chunk
// takes two to three times the tensor cores' cycles (busy for 39 % of a block's): each
// product waits for operands that another role makes from the one before it, and every
// wait or commit of the product warp costs 100 to 200 cycles, so that fewer of them, not
// fewer products, made it faster (training step 314 -> 295 us). Output rows go out as
// 32-byte stores of a head's 256 bytes; 16-byte stores were slower.
#include "scan_linattn_tc.h"
#include "scan_tc.cuh"

namespace scan {

namespace {

using namespace tc;

constexpr int kChunk = 128;
constexpr int kThreads = 18 * 32;  // four roles of four warps, a copy and a product warp
constexpr uint32_t kHalf = kChunk * kPitch;  // bytes of one panel of a chunk

struct TcPass {
  CUtensorMap x1, x2, x3;
  __nv_bfloat16* o;
  int64_t o_sb, o_st, o_sh;
  int o_wide;  // its rows start on 32 bytes and hold whole 32-byte pieces
  const float* s_in;
  float* s_out;
  float* seg;  // states after parts: dense [B][H][nseg - 1][pieces][K][V], packed [segments][H][K][V]
  float s_in_mul, s_out_mul;
  int s_in_t, K, V, reverse;
};

struct TcArgs {
  TcPass pass[3];
  const float* log_decay;
  const int32_t* cu;
  WsHeader* hdr;
  int64_t T;
  int npass, n_seqs, H;
  int nseg, cps, pieces;  // segments of a row, chunks of one, pieces in which its own state is found
  float scale;
};

template <int KP, int VP, bool STATE_ONLY>
struct Plan {
  static constexpr int kX1 = STATE_ONLY ? 0 : kChunk * 2 * KP;
  static constexpr int kX2 = kChunk * 2 * KP;
  static constexpr int kX3 = kChunk * 2 * VP;
  static constexpr int kStage = kX1 + kX2 + kX3;
  static constexpr int kState = STATE_ONLY ? 0 : VP * KP * 2;
  static constexpr int kTables = 2048;  // barriers, decay tables
  static constexpr int kFit = (232448 - 1024 - kTables - kState) / kStage;
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kSmem = kStages * kStage + kState + kTables + 1024;
};

// log2(lambda); no memory at all (-inf) as a number, so that its 0th power is 1. NaN
// stays NaN (which fmaxf would hide).
__device__ __forceinline__ float log2_decay(float log_decay) {
  const float l2 = log_decay * 1.44269504088896341f;
  return l2 < -1e30f ? -1e30f : l2;
}

// The part of the sequence that a block works on, in processing order.
struct Span {
  int64_t beg, len;  // the sequence
  int64_t first;     // first chunk of the segment, in processing order
  int nch;           // chunks of the segment, one at least
};

// Where the c-th chunk of the segment lies, and how many steps it holds.
__device__ __forceinline__ void chunk_at(const Span& s, bool reverse, int c, int64_t* t0, int* n) {
  const int64_t all = (s.len + kChunk - 1) / kChunk;
  const int64_t i = reverse ? all - 1 - (s.first + c) : s.first + c;
  *t0 = i * kChunk;
  const int64_t left = s.len - *t0;
  *n = (int)(left < kChunk ? left : kChunk);
}

template <int KP, int VP, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1) linattn_tc_kernel(const __grid_constant__ TcArgs a) {
  using P = Plan<KP, VP, STATE_ONLY>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;
  uint8_t* const gen = raw + (base - smem_addr(raw));
  // the passes of one part of a row run side by side: they read the same operands
  const unsigned item = blockIdx.x / a.npass;
  const TcPass& p = a.pass[blockIdx.x % a.npass];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

  // shared memory: stages, the state's bf16 copy, tables, barriers
  const uint32_t sState = base + P::kStages * P::kStage;
  float* const tab = reinterpret_cast<float*>(gen + P::kStages * P::kStage + P::kState);
  float* const wtab = tab;           // [128] weights of the update in a whole chunk
  float* const wlast = tab + 128;    // [128] in the chunk that ends the sequence, 0 past it
  // weights within a chunk, with the output's scale: [32] column powers, and [64] those of
  // row r and column c of a diagonal block, at 32 + r - c
  float* const ctab = tab + 256;
  float* const dtab = tab + 288;
  const uint32_t bars = smem_addr(tab + 352);
  const uint32_t bFull12 = bars, bFull3 = bars + 32, bFree12 = bars + 64, bFree3 = bars + 96, bS1 = bars + 128,
                 bP = bars + 136, bSb = bars + 144, bSt = bars + 152, bX = bars + 160, bXf = bars + 192,
                 bOi = bars + 224, bOs = bars + 232, bOf = bars + 240, bOx = bars + 248, bClean = bars + 256,
                 bInit = bars + 264;
  // places for 32 steps of the update's operand: half a chunk, or two whole ones
  constexpr int kBufs = STATE_ONLY ? 8 : 2;
  uint32_t* const tmem_ptr = reinterpret_cast<uint32_t*>(tab + 352) + 72;
  uint32_t* const stop_flag = tmem_ptr + 1;

  // which (sequence, head, segment): dense rows have nseg segments each; packed
  // sequences are cut into segments that are numbered through
  Span s{0, a.T, 0, 0};
  int h, seg = 0;
  int64_t sq, slot;  // slot: of the state after this part, among the workspace's
  bool last = true;  // the sequence's last segment
  if (a.cu) {
    h = (int)(item % a.H);
    const int64_t tile = item / a.H;
    int64_t e, local;
    int q;
    if (blockIdx.x == 0 && warp == 0 && !STATE_ONLY) check_seqlens(a.cu, a.n_seqs, a.T, a.hdr);
    if (!locate_tile(a.cu, a.n_seqs, a.T, tile, a.cps * kChunk, &s.beg, &e, &local, &q)) return;
    s.len = e - s.beg;
    sq = q;
    seg = (int)local;
    slot = tile * a.H + h;
    last = (local + 1) * a.cps * kChunk >= s.len;
    if (STATE_ONLY && last) return;
  } else {
    const int parts = STATE_ONLY ? (a.nseg - 1) * a.pieces : a.nseg;
    const int part = item % parts;
    const int64_t row = item / parts;
    h = (int)(row % a.H);
    sq = row / a.H;
    seg = STATE_ONLY ? part / a.pieces : part;
    slot = STATE_ONLY ? row * parts + part : (row * (a.nseg - 1) + seg + 1) * a.pieces - 1;
    last = seg == a.nseg - 1;
  }
  const int64_t row = sq * a.H + h;
  const int b = a.cu ? 0 : (int)sq;
  const int64_t all = (s.len + kChunk - 1) / kChunk;
  if (STATE_ONLY && !a.cu) {
    const int i = item % a.pieces, c0 = a.cps * i / a.pieces;
    s.first = (int64_t)seg * a.cps + c0;
    s.nch = a.cps * (i + 1) / a.pieces - c0;
  } else {
    s.first = (int64_t)seg * a.cps;
    s.nch = (int)(all - s.first < a.cps ? all - s.first : a.cps);
  }
  const bool rev = p.reverse != 0;
  // steps of this part: chunks are whole but the one that ends the sequence
  const int64_t steps = s.nch * (int64_t)kChunk -
                        ((rev ? s.first == 0 : s.first + s.nch == all) ? all * kChunk - s.len : 0);
  const int e = rev ? 0 : 1;
  const float l2 = log2_decay(a.log_decay[h]);

  // initial state: the caller's for the first segment, else the one before
  const float* s0 = nullptr;
  int s0k = 0, s0v = 0;  // its strides
  float s0m = 1.f;
  if (s.first == 0) {
    if (p.s_in) {
      s0 = p.s_in + row * p.K * p.V;
      s0k = p.s_in_t ? 1 : p.V;
      s0v = p.s_in_t ? p.K : 1;
      s0m = p.s_in_mul;
    }
  } else if (!STATE_ONLY) {
    s0 = p.seg + (a.cu ? slot - a.H : slot - a.pieces) * p.K * p.V;
    s0k = p.V;
    s0v = 1;
  }
  // final state: after a segment, or the caller's after the last
  float* s1 = nullptr;
  float s1m = 1.f;
  if (STATE_ONLY) {
    s1 = p.seg + slot * p.K * p.V;
  } else if (last && p.s_out) {
    s1 = p.s_out + row * p.K * p.V;
    s1m = p.s_out_mul;
  }
  const bool packed = a.cu != nullptr;
  const int late = s0 ? 0 : 1;  // the first chunk whose queries read a state

  // one chunk of x1, x2 and x3 into its stage
  const auto load12 = [&](int c) {
    int64_t t0;
    int n;
    chunk_at(s, rev, c, &t0, &n);
    const int st = c % P::kStages, t = (int)(s.beg + t0);
    const uint32_t d = base + st * P::kStage;
    bar_expect(bFull12 + 8 * st, P::kX1 + P::kX2);
#pragma unroll
    for (int i = 0; i < KP / 64; ++i) {
      if (!STATE_ONLY) copy_in_4d(d + i * kHalf, &p.x1, bFull12 + 8 * st, 64 * i, h, t, b);
      copy_in_4d(d + P::kX1 + i * kHalf, &p.x2, bFull12 + 8 * st, 64 * i, h, t, b);
    }
  };
  const auto load3 = [&](int c) {
    int64_t t0;
    int n;
    chunk_at(s, rev, c, &t0, &n);
    const int st = c % P::kStages, t = (int)(s.beg + t0);
    bar_expect(bFull3 + 8 * st, P::kX3);
#pragma unroll
    for (int i = 0; i < VP / 64; ++i)
      copy_in_4d(base + st * P::kStage + P::kX1 + P::kX2 + i * kHalf, &p.x3, bFull3 + 8 * st, 64 * i, h, t, b);
  };
  // the copy warp sets the barriers up and fills the stages while the others prepare
  if (warp == 16 && lane == 0) {
    *stop_flag = 0;
    for (int i = 0; i < P::kStages; ++i) {
      bar_init(bFull12 + 8 * i, 1);
      bar_init(bFull3 + 8 * i, 1);
      bar_init(bFree12 + 8 * i, 1);
      bar_init(bFree3 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(bX + 8 * i, STATE_ONLY ? 16 : 4);
      bar_init(bXf + 8 * i, 1);
    }
    bar_init(bS1, 1);
    bar_init(bP, 4);
    bar_init(bSb, 4);
    bar_init(bSt, 1);
    bar_init(bOi, 1);
    bar_init(bOs, 4);
    bar_init(bOf, 1);
    bar_init(bOx, 4);
    bar_init(bClean, STATE_ONLY ? 16 : 4);  // every warp that clears rows of the next sequence
    bar_init(bInit, 4 * (KP / 32));
    bar_init_fence();
    for (int c = 0; c < P::kStages && c < s.nch; ++c) {
      load12(c);
      load3(c);
    }
  }
  __syncwarp();
  if (tid < 128) {
    const int n = s.len % kChunk ? (int)(s.len % kChunk) : kChunk;
    wtab[tid] = exp2f(l2 * (float)(rev ? tid + 1 : 127 - tid));
    wlast[tid] = tid < n ? exp2f(l2 * (float)(rev ? tid + 1 : n - 1 - tid)) : 0.f;
  }
  if (tid < 64) {
    const int d = rev ? 32 - tid : tid - 32;
    dtab[tid] = d >= 0 ? a.scale * exp2f(l2 * (float)d) : 0.f;
  }
  if (tid < 32) ctab[tid] = a.scale * exp2f(l2 * (float)(rev ? tid : 31 - tid));
  if (warp == 17) tmem_alloc(smem_addr(tmem_ptr), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = *tmem_ptr;
  // tensor memory: S1 (P over its first half), the update's pieces of 32 steps (two or
  // three bf16 parts of 16 columns each), O, S^T
  const uint32_t tS1 = tm, tX = STATE_ONLY ? tm : tm + 128, tO = tm + 256, tSt = tm + 384;
  constexpr int kPiece = 48;
  // two parts carry the state to 2^-16 a step, which the bf16 outputs never show; a
  // state that is an output itself gets three
  const bool three = p.s_out != nullptr;
  const uint32_t lanes = (uint32_t)(warp % 4) << 21;  // this warp's first tensor-memory lane
  const Stop stop{stop_flag, a.hdr};
  const int role = warp / 4;

  // 32 rows of S to its bf16 copy, and decayed to tensor memory
  const auto give = [&](uint32_t(&r)[32], int kb, float keep) {
    const int v = tid % 128;
    if (!STATE_ONLY && v < VP) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t o[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
          o[x] = pack_bf16(__uint_as_float(r[8 * y + 2 * x]), __uint_as_float(r[8 * y + 2 * x + 1]));
        st_shared16(swizzled(sState + (kb / 2) * VP * kPitch, v, (kb % 2) * 4 + y), o[0], o[1], o[2], o[3]);
      }
    }
#pragma unroll
    for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * keep);
    tmem_st32(tSt + lanes + 32 * kb, r);
  };
  if (!STATE_ONLY && s0 && role < KP / 32) {
    // the state that comes in: 32 of its rows a role, all loads in flight at once
    const int v = tid % 128;
    int64_t t0;
    int n;
    chunk_at(s, rev, 0, &t0, &n);
    uint32_t r[32];
#pragma unroll
    for (int x = 0; x < 32; ++x) {
      const int k = 32 * role + x;
      r[x] = __float_as_uint(s0[(k < p.K ? k : 0) * s0k + (v < p.V ? v : 0) * s0v]);
    }
#pragma unroll
    for (int x = 0; x < 32; ++x)
      r[x] = v < p.V && 32 * role + x < p.K ? __float_as_uint(s0m * __uint_as_float(r[x])) : 0u;
    give(r, role, exp2f(l2 * (float)n));
    st_wait();
    fence_async();
    fence_before();
    __syncwarp();
    if (lane == 0) bar_arrive(bInit);
    __syncwarp();
  }

  if (warp == 16) {
    // ---- copies
    if (lane == 0) {
      for (int c = P::kStages; c < s.nch; ++c) {
        const int st = c % P::kStages;
        const uint32_t again = (c / P::kStages - 1) & 1;
        if (!bar_wait(bFree12 + 8 * st, again, stop)) break;
        load12(c);
        if (!bar_wait(bFree3 + 8 * st, again, stop)) break;
        load3(c);
      }
    }
  } else if (warp == 17) {
    // ---- products
    {
      const bool lead = lane == 0;
      constexpr uint32_t dS1 = product_desc(128, 128, false, false);
      constexpr uint32_t dOi = product_desc(128, VP, false, false);
      constexpr uint32_t dSt = product_desc(128, KP, false, true);
      constexpr uint32_t dO = product_desc(128, VP, false, true);
      const auto ready = [&](int c) {  // chunk c has arrived, and nothing in it is another sequence's
        int64_t t0;
        int n;
        chunk_at(s, rev, c, &t0, &n);
        return warp_wait(bFull12 + 8 * (c % P::kStages), (c / P::kStages) & 1, stop) &&
               (!packed || n == kChunk || warp_wait(bClean, 0, stop));
      };
      const auto scores = [&](int c) {
        const uint32_t x1 = kmajor(base) + (c % P::kStages) * (P::kStage >> 4);
        mma_kk<KP, kHalf, kHalf>(lead, tS1, x1, x1 + (P::kX1 >> 4), dS1, false);
        mma_commit(lead, bS1);
      };
      bool ok = true;
      if (!STATE_ONLY && (ok = ready(0))) scores(0);
#pragma unroll 1
      for (int c = 0; ok && c < s.nch; ++c) {
        const int st = c % P::kStages;
        const uint32_t x1 = kmajor(base) + st * (P::kStage >> 4);
        const uint32_t x2 = mnmajor(base + P::kX1, kHalf) + st * (P::kStage >> 4), x3 = x2 + (P::kX2 >> 4);
        const bool have = c > 0 || (s0 && !STATE_ONLY);
        if (STATE_ONLY) ok = ready(c);
        else if (c > 0) ok = warp_wait(bSb, (c - 1) & 1, stop);
        else if (s0) ok = warp_wait(bInit, 0, stop);
        if (!ok) break;
        fence_after();
        // Each wait or commit of this warp costs the tensor cores 100 to 200 cycles, so
        // what a role hands over also says that the copies it has waited for are there,
        // and roles give operands back. The update's operand comes in halves of a chunk;
        // the second waits for the first to be used, so the state is read in between.
        const bool more = c + 1 < s.nch || s1;
        const auto piece = [&](int jb, uint32_t at) {
          mma_tn<32>(lead, tSt, at, x2 + jb * (32 * kPitch >> 4), dSt, have || jb > 0);
          mma_tn<32>(lead, tSt, at + 16, x2 + jb * (32 * kPitch >> 4), dSt, true);
          if (three) mma_tn<32>(lead, tSt, at + 32, x2 + jb * (32 * kPitch >> 4), dSt, true);
        };
        if (STATE_ONLY) {
          const int set = c & 1;
          if (!(ok = warp_wait(bX + 8 * set, (c >> 1) & 1, stop))) break;
          fence_after();
#pragma unroll
          for (int jb = 0; jb < 4; ++jb) piece(jb, tX + kPiece * (4 * set + jb));
          mma_commit(lead, bXf + 8 * set);
          mma_commit(lead, bFree12 + 8 * st);
          mma_commit(lead, bFree3 + 8 * st);
          if (c + 1 == s.nch) mma_commit(lead, bSt);
          continue;
        }
        if (more) {
          if (!(ok = warp_wait(bX, c & 1, stop))) break;
          fence_after();
          piece(0, tX);
          piece(1, tX + kPiece);
          mma_commit(lead, bXf);
        }
        if (c > 0 && !(ok = warp_wait(bOx, (c - 1) & 1, stop))) break;
        fence_after();
        if (have) {
          mma_kk<KP, kHalf, VP * kPitch>(lead, tO, x1, kmajor(sState), dOi, false);
          mma_commit(lead, bOi);
        }
        if (more) {
          if (!(ok = warp_wait(bX + 8, c & 1, stop))) break;
          fence_after();
          piece(2, tX);
          piece(3, tX + kPiece);
        } else if (!(ok = warp_wait(bFull3 + 8 * st, (c / P::kStages) & 1, stop))) {
          break;
        }
        mma_commit(lead, bSt);
        if (!(ok = warp_wait(bP, c & 1, stop))) break;
        if (have && !(ok = warp_wait(bOs, (c - late) & 1, stop))) break;
        fence_after();
        mma_tn<kChunk>(lead, tO, tS1, x3, dO, have);
        mma_commit(lead, bOf);
        if (c + 1 < s.nch) scores(c + 1);  // over P, which the product before has read
      }
    }
  } else if (role == 0 && !STATE_ONLY) {
    // ---- weights: row i of the chunk in lane i. Blocks of 32 columns before
    // (reversed: after) the warp's own rows factor into a row and a column power
    // of lambda that are both at most 1; the diagonal block takes the power of
    // the difference.
    const int w = warp % 4;
#pragma unroll 1
    for (int c = 0; c < s.nch; ++c) {
      if (!warp_wait(bS1, c & 1, stop)) break;
      fence_after();
#pragma unroll 1
      for (int jb = 0; jb < 4; ++jb) {  // (rolled: the four roles' code has to fit the instruction cache)
        uint32_t o[16];
        if (rev ? jb < w : jb > w) {
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] = 0;
        } else {
          uint32_t r[32];
          tmem_ld32(tS1 + lanes + 32 * jb, r);
          ld_wait();
          if (jb == w) {
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const float2 f = mul2(pair_of(r + x), make_float2(dtab[32 + lane - x], dtab[31 + lane - x]));
              o[x / 2] = pack_bf16(f.x, f.y);
            }
          } else {
            const float f = exp2f(l2 * (float)(rev ? 32 * (jb - w) - lane : 32 * (w - jb) + lane - 31));
            const float2 rf = make_float2(f, f);
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 k = *reinterpret_cast<const float4*>(ctab + x);
              const float2 f0 = mul2(pair_of(r + x), mul2(rf, make_float2(k.x, k.y)));
              const float2 f1 = mul2(pair_of(r + x + 2), mul2(rf, make_float2(k.z, k.w)));
              o[x / 2] = pack_bf16(f0.x, f0.y);
              o[x / 2 + 1] = pack_bf16(f1.x, f1.y);
            }
          }
        }
        tmem_st16(tS1 + lanes + 16 * jb, o);  // over columns that have been read
      }
      st_wait();
      fence_before();
      if (w == 0 && c + 1 < s.nch) {  // the next chunk's x1 and x2 are there
        int64_t t0;
        int n;
        chunk_at(s, rev, c + 1, &t0, &n);
        if (!warp_wait(bFull12 + 8 * ((c + 1) % P::kStages), ((c + 1) / P::kStages) & 1, stop)) break;
        if (packed && n < kChunk && !warp_wait(bClean, 0, stop)) break;
      }
      __syncwarp();
      if (lane == 0) bar_arrive(bP);
    }
  } else if (role == 1 && !STATE_ONLY) {
    // ---- state: column v of S (a row of S^T) in lane v
#pragma unroll 1
    for (int c = 1; c < s.nch; ++c) {
      int64_t t0;
      int n;
      chunk_at(s, rev, c, &t0, &n);
      const float keep = exp2f(l2 * (float)n);
      if (!warp_wait(bSt, (c - 1) & 1, stop)) break;
      fence_after();
      if (warp == 4 && lane == 0) bar_arrive(bFree12 + 8 * ((c - 1) % P::kStages));  // all their products are done
      __syncwarp();
#pragma unroll 1
      for (int kb = 0; kb < KP / 32; ++kb) {
        uint32_t r[32];
        tmem_ld32(tSt + lanes + 32 * kb, r);
        ld_wait();
        give(r, kb, keep);
      }
      st_wait();
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(bSb);
    }
  } else if (role == 2 || (STATE_ONLY && role < 4)) {
    // ---- update: column v of x3 in lane v, weighted and split in two, 32 steps at a
    // time (by all four roles, each a quarter, where only the state is wanted)
    const int v = tid % 128;
    if (v >= VP) {  // lanes past V: zeros, once
      uint32_t z[32];
#pragma unroll
      for (int x = 0; x < 32; ++x) z[x] = 0;
#pragma unroll
      for (int x = 0; x < kBufs * kPiece / 32; ++x) tmem_st32(tX + lanes + 32 * x, z);
      st_wait();
    }
    bool ok = true;
#pragma unroll 1
    for (int c = 0; ok && c < s.nch; ++c) {
      const int st = c % P::kStages;
      int64_t t0;
      int n;
      chunk_at(s, rev, c, &t0, &n);
      if (!warp_wait(bFull3 + 8 * st, (c / P::kStages) & 1, stop)) break;
      if (packed && n < kChunk) {
        if (!warp_wait(bFull12 + 8 * st, (c / P::kStages) & 1, stop)) break;
        // the rows from n on belong to the next sequence (one such chunk a row)
        const uint32_t x2 = base + st * P::kStage + P::kX1;
        const int left = kChunk - n;
        for (int i = v; i < left * 8 * (KP + VP) / 64; i += 128) {
          const int piece = i % 8, r = n + (i / 8) % left, pn = i / 8 / left;
          st_shared16(x2 + pn * kHalf + r * kPitch + piece * 16, 0, 0, 0, 0);
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(bClean);
        __syncwarp();
        if (!warp_wait(bClean, 0, stop)) break;
      }
      if (!(c + 1 < s.nch || s1)) break;  // no one reads the state after this chunk
      const uint8_t* col = gen + st * P::kStage + P::kX1 + P::kX2 + (v < VP ? v / 64 : 0) * kHalf + (v % 8) * 2;
      const int piece = (v % 64) / 8;
      const float* wt = n < kChunk ? wlast : wtab;
      // a segment on its own: weights to its end, the sums never rescaled
      const float far = STATE_ONLY ? exp2f(l2 * (float)((s.nch - 1 - c) * kChunk)) : 1.f;
#pragma unroll 1
      for (int jb = STATE_ONLY ? role : 0; jb < 4; jb += STATE_ONLY ? 4 : 1) {
        uint32_t hi[16], mid[16], lo[16];
        if (v < VP) {
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            const float4 w4 = *reinterpret_cast<const float4*>(wt + 32 * jb + 2 * x);
            const float w[4] = {w4.x * far, w4.y * far, w4.z * far, w4.w * far};
            float f[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const int j = 2 * x + y;
              const uint32_t u =
                  *reinterpret_cast<const uint16_t*>(col + 32 * jb * kPitch + j * kPitch + ((piece ^ (j & 7)) << 4));
              f[y] = __uint_as_float(u << 16) * w[y];
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t h = pack_bf16(f[2 * y], f[2 * y + 1]);
              const float g0 = f[2 * y] - __uint_as_float(h << 16);
              const float g1 = f[2 * y + 1] - __uint_as_float(h & 0xffff0000u);
              const uint32_t m = pack_bf16(g0, g1);
              hi[x + y] = h;
              mid[x + y] = m;
              if (three) lo[x + y] = pack_bf16(g0 - __uint_as_float(m << 16), g1 - __uint_as_float(m & 0xffff0000u));
            }
          }
        }
        // the place's last use is over
        if (STATE_ONLY) ok = c < 2 || warp_wait(bXf + 8 * (c & 1), ((c >> 1) - 1) & 1, stop);
        else if (jb == 0) ok = c == 0 || warp_wait(bSt, (c - 1) & 1, stop);
        else if (jb == 2) ok = warp_wait(bXf, c & 1, stop);
        if (!ok) break;
        fence_after();
        const uint32_t at = tX + kPiece * (STATE_ONLY ? 4 * (c & 1) + jb : jb & 1) + lanes;
        if (v < VP) {
          tmem_st16(at, hi);
          tmem_st16(at + 16, mid);
          if (three) tmem_st16(at + 32, lo);
          st_wait();
        }
        if (STATE_ONLY || (jb & 1)) {
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(bX + 8 * (STATE_ONLY ? c & 1 : jb >> 1));
          __syncwarp();
        }
      }
    }
  } else if (role == 3 && !STATE_ONLY) {
    // ---- output: row i of the chunk in lane i
    const int i = tid - 384;
#pragma unroll 1
    for (int c = 0; c < s.nch; ++c) {
      int64_t t0;
      int n;
      chunk_at(s, rev, c, &t0, &n);
      if (c > 0 || s0) {
        if (!warp_wait(bOi, (c - late) & 1, stop)) break;
        fence_after();
        const int r = rev ? n - 1 - i : i;
        const float f = r >= 0 ? a.scale * exp2f(l2 * (float)(r + e)) : 0.f;
#pragma unroll 1
        for (int vb = 0; vb < VP / 32; ++vb) {
          uint32_t x[32];
          tmem_ld32(tO + lanes + 32 * vb, x);
          ld_wait();
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * f);
          tmem_st32(tO + lanes + 32 * vb, x);
        }
        st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(bOs);
      }
      if (!warp_wait(bOf, c & 1, stop)) break;
      fence_after();
      if (i == 0) bar_arrive(bFree3 + 8 * (c % P::kStages));
      __syncwarp();
      __nv_bfloat16* const orow = p.o + b * p.o_sb + (s.beg + t0 + i) * p.o_st + h * p.o_sh;
#pragma unroll 1
      for (int vb = 0; vb < VP / 32; ++vb) {
        uint32_t x[32], o[16];
        tmem_ld32(tO + lanes + 32 * vb, x);
        ld_wait();
        if (vb == VP / 32 - 1) {  // O may be written again
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(bOx);
          __syncwarp();
        }
#pragma unroll
        for (int y = 0; y < 16; ++y) o[y] = pack_bf16(__uint_as_float(x[2 * y]), __uint_as_float(x[2 * y + 1]));
        // whole 32-byte sectors a lane where the rows allow
#pragma unroll
        for (int y = 0; y < 16; y += 8) {
          const int col = 32 * vb + 2 * y;
          if (i < n && p.o_wide) {
            if (col < p.V) st_global32(orow + col, o + y);
          } else if (i < n) {
            if (col < p.V) *reinterpret_cast<uint4*>(orow + col) = make_uint4(o[y], o[y + 1], o[y + 2], o[y + 3]);
            if (col + 8 < p.V)
              *reinterpret_cast<uint4*>(orow + col + 8) = make_uint4(o[y + 4], o[y + 5], o[y + 6], o[y + 7]);
          }
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  if (role == 1 && s1) {
    // ---- the final state, by the state's role: column v in lane v
    const int v = tid % 128;
    if (warp_wait(bSt, STATE_ONLY ? 0 : (s.nch - 1) & 1, stop)) {
      fence_after();
      // a segment on its own starts from nothing: what came in is added here
      const float in = s0m * exp2f(l2 * (float)steps);
      const bool add = STATE_ONLY && s0;
      const bool on = v < p.V;
      const float* const si = add ? s0 + (on ? v : 0) * s0v : nullptr;
      float* const so = s1 + v;
#pragma unroll 1
      for (int kb = 0; kb < KP / 32; ++kb) {
        uint32_t r[32];
        tmem_ld32(tSt + lanes + 32 * kb, r);
        ld_wait();
        if (add) {
          float f[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) f[x] = si[(32 * kb + x < p.K ? 32 * kb + x : 0) * s0k];
#pragma unroll
          for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(fmaf(in, f[x], __uint_as_float(r[x])));
        }
#pragma unroll
        for (int x = 0; x < 32; x += 8) {  // K is a multiple of 8
          if (on && 32 * kb + x < p.K) {
#pragma unroll
            for (int y = 0; y < 8; ++y) so[(32 * kb + x + y) * p.V] = s1m * __uint_as_float(r[x + y]);
          }
        }
      }
    }
  }
  __syncwarp();
  linger(stop);
  fence_before();
  __syncthreads();
  if (warp == 17) {
    fence_after();
    tmem_free(tm, 512);
  }
}

// The states after parts, from each part's own: S_i = lambda^steps S_(i-1) + own_i;
// the parts are a dense row's pieces, or a packed sequence's segments but its last
// (of whole chunks all but the row's first, which adds to nothing). An empty packed
// sequence has no part of the row; its final state is written here.
__global__ void __launch_bounds__(256) linattn_chain_kernel(const __grid_constant__ TcArgs a) {
  const TcPass& p = a.pass[blockIdx.z];
  const int n = p.K * p.V;  // a multiple of 64
  const int64_t row = blockIdx.x;  // (there may be more rows than a grid's other axes hold)
  const int i = (blockIdx.y * 256 + threadIdx.x) * 4;
  const int h = (int)(row % a.H), seq = (int)(row / a.H);
  const float l2 = log2_decay(a.log_decay[h]);
  __shared__ float keep[64];  // lambda^steps of a dense segment's pieces
  if (!a.cu && threadIdx.x < a.pieces) {
    const int y = threadIdx.x, chunks = a.cps * (y + 1) / a.pieces - a.cps * y / a.pieces;
    keep[y] = exp2f(l2 * (float)(chunks * kChunk));
  }
  __syncthreads();
  int count = (a.nseg - 1) * a.pieces;
  int64_t first = row * count, step = 1;
  float whole = 1.f;
  if (a.cu) {
    int64_t beg, end, before = 0;  // segments of the sequences before this one
    for (int q = threadIdx.x % 32; q < seq; q += 32) {
      seq_bounds(a.cu, q, a.T, &beg, &end);
      before += (end - beg + a.cps * kChunk - 1) / (a.cps * kChunk);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
    seq_bounds(a.cu, seq, a.T, &beg, &end);
    count = (int)((end - beg + a.cps * kChunk - 1) / (a.cps * kChunk)) - 1;
    // offsets that overlap (malformed) add up to more segments than the workspace holds
    if (before + count > a.nseg) count = 0;
    first = before * a.H + h;
    step = a.H;
    whole = exp2f(l2 * (float)(a.cps * kChunk));
    if (count < 0 && p.s_out) {
      for (int j = i; j < i + 4 && j < n; ++j) {
        const int k = j / p.V, v = j % p.V;
        p.s_out[row * n + j] = !p.s_in ? 0.f : p.s_out_mul * p.s_in_mul * p.s_in[row * n + (p.s_in_t ? v * p.K + k : j)];
      }
    }
  }
  if (i >= n || count < 2) return;
  float4* s = reinterpret_cast<float4*>(p.seg + first * n + i);
  const int64_t by = step * n / 4;
  float4 acc = s[0];
  int y = 0;
  for (int g = 1; g < count; g += 4) {  // four loads at a time
    float4 own[4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (g + x < count) own[x] = s[(g + x) * by];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (g + x >= count) break;
      y = y + 1 == a.pieces ? 0 : y + 1;
      const float f = a.cu ? whole : keep[y];
      acc.x = fmaf(f, acc.x, own[x].x);
      acc.y = fmaf(f, acc.y, own[x].y);
      acc.z = fmaf(f, acc.z, own[x].z);
      acc.w = fmaf(f, acc.w, own[x].w);
      s[(g + x) * by] = acc;
    }
  }
}

struct Split {
  int nseg, cps, pieces;
};

// Segments of a row, by the time that they would take in chunks of one block (152
// blocks at a time, two chunks for a block's start and end): more segments fill the
// SMs and shorten what one block does, but their own states have to be found first
// from a second read of x2 and x3 (half a chunk's time each, in pieces that fill the
// SMs as well; three chunks for the two launches). `rows` are the (sequence, head)
// rows of all passes.
Split split_rows(int64_t rows, int64_t T) {
  const int64_t nch = (T + kChunk - 1) / kChunk;
  Split best{1, (int)nch, 1};
  if (rows <= 0) return best;
  const auto rounds = [](int64_t blocks) { return (double)((blocks + 151) / 152); };
  double least = rounds(rows) * (double)(nch + 2);
  for (int64_t n = 2; n <= 32 && n <= nch / 2; ++n) {
    const int64_t cps = (nch + n - 1) / n, used = (nch + cps - 1) / cps;
    if (used != n) continue;
    for (int64_t m = 1; m <= 8 && m <= cps; ++m) {
      const double own = rounds(rows * (n - 1) * m) * (double)((cps + m - 1) / m + 2) * 0.5;
      const double time = rounds(rows * n) * (double)(cps + 2) + own + 3.0;
      if (time < least) {
        least = time;
        best = Split{(int)n, (int)cps, (int)m};
      }
    }
  }
  return best;
}
// Packed sequences, whose lengths the host does not know: segments of one size,
// such that the row's own number of them, and half a segment more a sequence, fill
// the SMs once; at least four chunks each. nseg: segments of a head at most.
Split split_packed(int64_t n_seqs, int64_t H, int64_t T) {
  const int64_t nch = (T + kChunk - 1) / kChunk;
  int64_t want = H > 0 ? 152 / H - n_seqs / 2 : 1;
  want = want < 1 ? 1 : want;
  int64_t cps = (nch + want - 1) / want;
  cps = cps < 4 ? 4 : cps > 1 << 20 ? 1 << 20 : cps;  // a segment's steps are 32-bit numbers
  return Split{(int)((nch + cps - 1) / cps + n_seqs), (int)cps, 1};
}
// A row of one segment's length has none to chain, however its sequences lie.
bool packed_chains(const Split& sp, int64_t T) { return (int64_t)sp.cps * kChunk < T; }

int padded(int d) { return d <= 64 ? 64 : 128; }

template <int KP, int VP>
cudaError_t launch_kv(const TcArgs& t, int npass, int64_t rows, cudaStream_t s) {
  using P = Plan<KP, VP, false>;
  using Q = Plan<KP, VP, true>;
  static_assert(P::kSmem <= 232448 && P::kStages >= 2 && Q::kSmem <= 232448, "fits a block's shared memory");
  cudaError_t e = cudaFuncSetAttribute(linattn_tc_kernel<KP, VP, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
  if (e != cudaSuccess) return e;
  // (a packed row without segments to chain may have empty sequences)
  const bool split = t.cu ? packed_chains(Split{t.nseg, t.cps, t.pieces}, t.T) : t.nseg > 1;
  const int64_t own = t.cu ? (int64_t)t.nseg * t.H : rows * (t.nseg - 1) * t.pieces;
  const int64_t parts = t.cu ? (int64_t)t.nseg * t.H : rows * t.nseg;
  if (split) {
    e = cudaFuncSetAttribute(linattn_tc_kernel<KP, VP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Q::kSmem);
    if (e != cudaSuccess) return e;
    linattn_tc_kernel<KP, VP, true><<<(unsigned)(own * npass), kThreads, Q::kSmem, s>>>(t);
  }
  if (split || t.cu)
    linattn_chain_kernel<<<dim3((unsigned)rows, KP * VP / 1024, npass), 256, 0, s>>>(t);
  linattn_tc_kernel<KP, VP, false><<<(unsigned)(parts * npass), kThreads, P::kSmem, s>>>(t);
  return cudaGetLastError();
}

cudaError_t launch_passes(const TcArgs& t, int npass, int64_t rows, cudaStream_t s) {
  const int K = padded(t.pass[0].K), V = padded(t.pass[0].V);
  if (K == 64 && V == 64) return launch_kv<64, 64>(t, npass, rows, s);
  if (K == 64) return launch_kv<64, 128>(t, npass, rows, s);
  if (V == 64) return launch_kv<128, 64>(t, npass, rows, s);
  return launch_kv<128, 128>(t, npass, rows, s);
}

}  // namespace

// bf16 operands that tensor copies can address, and rows long enough that a
// chunk's fixed chain of products is shorter than the recurrence.
bool linattn_tc_fits(const LinArgs& a, scan_dtype dt) {
  if (dt != SCAN_BF16 || a.T < 1 || a.T > 0x7fffffffLL) return false;
  const int64_t n = a.cu ? a.n_seqs : a.B;
  // Rows of fewer steps go one step at a time. A row's chunk costs the same whatever it
  // holds and whatever its heads are padded to; a step's cost follows the head. Forward,
  // us by chunks / by steps, for 16 and 1024 (sequence, head) rows:
  //   128 x 128:  8 steps 5.5 / 7.1 and 33 / 50,   16 steps 5.7 / 11 and 32 / 87
  //    64 x 64:   8 steps 5.1 / 5.2 and 28 / 16,   16 steps 4.9 / 7.9 and 28 / 26
  //    32 x 32:  16 steps 5.1 / 7.8 and 28 / 14,   32 steps 5.1 / 14 and 28 / 25
  // so that small heads in more rows than three rounds of blocks have a bound of their own
  // (their backward, 1024 rows: 24 steps 79 / 53, 32 steps 78 / 67, 40 steps 79 / 83).
  const bool small = a.pass[0].K <= 32 && a.pass[0].V <= 32 && n * a.H * a.npass > 3 * 152;
  if (a.T < (small ? 32 : 16) * (a.cu ? n : 1)) return false;
  for (int i = 0; i < a.npass; ++i) {
    const LinPass& p = a.pass[i];
    if (!heads_map_fits(p.x1, a.B, a.T, a.H) || !heads_map_fits(p.x2, a.B, a.T, a.H) ||
        !heads_map_fits(p.x3, a.B, a.T, a.H) || !heads_map_fits(p.out, a.B, a.T, a.H))
      return false;
  }
  return true;
}

size_t linattn_tc_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t Dk, int64_t Dv,
                                  int64_t n_seqs) {
  int64_t slots = 0;  // of all passes: three backward, one forward
  if (n_seqs > 0) {
    const Split sp = split_packed(n_seqs, H, T);
    slots = packed_chains(sp, T) ? 3 * (int64_t)sp.nseg * H : 0;
  } else {
    for (int passes = 1; passes <= 3; passes += 2) {
      const Split sp = split_rows(B * H * passes, T);
      const int64_t need = passes * B * H * (sp.nseg - 1) * sp.pieces;
      slots = need > slots ? need : slots;
    }
  }
  return (size_t)(slots * Dk * Dv) * 4;
}

cudaError_t launch_linattn_tc(const LinArgs& a, cudaStream_t s) {
  const int64_t n = a.cu ? a.n_seqs : a.B, rows = n * a.H;
  const Split sp = a.cu ? split_packed(a.n_seqs, a.H, a.T) : split_rows(rows * a.npass, a.T);
  const int64_t slots = a.cu ? (int64_t)sp.nseg * a.H : rows * (sp.nseg - 1) * sp.pieces;
  TcArgs t[2];
  int count[2] = {0, 0};
  for (int i = 0; i < a.npass; ++i) {
    const LinPass& p = a.pass[i];
    // passes of one padded shape go in one launch
    const int g = i > 0 && (padded(p.K) != padded(a.pass[0].K) || padded(p.V) != padded(a.pass[0].V));
    TcPass& d = t[g].pass[count[g]++];
    if (!encode_heads_map(&d.x1, p.x1, a.B, a.T, a.H, p.K, kChunk) ||
        !encode_heads_map(&d.x2, p.x2, a.B, a.T, a.H, p.K, kChunk) ||
        !encode_heads_map(&d.x3, p.x3, a.B, a.T, a.H, p.V, kChunk))
      return cudaErrorInvalidValue;
    d.o = static_cast<__nv_bfloat16*>(p.out.ptr);
    d.o_sb = p.out.stride_b;
    d.o_st = p.out.stride_t;
    d.o_sh = p.out.stride_h;
    d.o_wide = (uintptr_t)p.out.ptr % 32 == 0 && p.V % 16 == 0 && (a.B == 1 || d.o_sb % 16 == 0) &&
               (a.T == 1 || d.o_st % 16 == 0) && (a.H == 1 || d.o_sh % 16 == 0);
    d.s_in = p.s_in;
    d.s_out = p.s_out;
    d.s_in_mul = p.s_in_mul;
    d.s_out_mul = p.s_out_mul;
    d.s_in_t = p.s_in_t;
    d.K = p.K;
    d.V = p.V;
    d.reverse = p.reverse;
    d.seg = a.ws + (int64_t)i * slots * p.K * p.V;
  }
  for (int g = 0; g < 2; ++g) {
    if (!count[g]) continue;
    t[g].npass = count[g];
    t[g].log_decay = a.log_decay;
    t[g].cu = a.cu;
    t[g].hdr = a.hdr;
    t[g].T = a.T;
    t[g].n_seqs = a.n_seqs;
    t[g].H = a.H;
    t[g].nseg = sp.nseg;
    t[g].cps = sp.cps;
    t[g].pieces = sp.pieces;
    t[g].scale = a.scale;
    const cudaError_t e = launch_passes(t[g], count[g], rows, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace scan
