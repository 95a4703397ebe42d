// scan_philox.cuh -- random numbers from a counter: Philox 4x32 with ten rounds
// (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011). The 128-bit counter is (block, call), the 64-bit key the seed. A
// number depends on nothing else, so that a backward pass, or the same call on
// other hardware shapes, draws it again instead of reading it.
#pragma once

#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

namespace scan {

// The four words of block `block`. A round is two 32 x 32 -> 64 bit products and two
// three-way exclusive ors; ten rounds are some sixty instructions.
__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t call, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)call, c3 = (uint32_t)(call >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Dropout with probability p in steps of 2^-16: of the eight 16-bit numbers of a
// block, element i of the tensor has number i % 8 of block i / 8 (low half of a word
// first), and is dropped where that is below `limit`. What stays is multiplied by
// 65536 / (65536 - limit), so the mean is kept exactly for the p that is applied. 16
// bits an element halve the generator's work against 32; p is off by 2^-17 at most.
struct Drop {
  uint32_t limit;       // 0: nothing is dropped
  uint32_t above;       // 65536 limit - 1: what a number's 16 bits, as a word's upper ones, have to pass
  float scale;
  uint64_t seed, call;  // used where rng is null
  const int64_t* rng;   // nullable: {seed, call} on the device
  __device__ __forceinline__ void read(uint64_t* s, uint64_t* c) const {
    *s = rng ? (uint64_t)rng[0] : seed;
    *c = rng ? (uint64_t)rng[1] : call;
  }
};

inline Drop make_drop(double p, uint64_t seed, uint64_t call, const int64_t* rng) {
  Drop d{};
  d.limit = (uint32_t)nearbyint(p * 65536.0);  // 0 <= p <= 1; ties to even
  d.above = (uint32_t)(((uint64_t)d.limit << 16) - 1);
  d.scale = d.limit < 65536u ? (float)(65536.0 / (65536.0 - d.limit)) : 0.f;
  d.seed = seed;
  d.call = call;
  d.rng = rng;
  return d;
}

// The eight elements of a block times what they are kept with. An element that is dropped
// is 0 whatever it holds. (limit > 0)
__device__ __forceinline__ void drop8(float2 (&v)[4], const Drop& d, uint64_t block, uint64_t call, uint64_t seed) {
  const uint4 r = philox(block, call, seed);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i].x = w[i] << 16 > d.above ? v[i].x * d.scale : 0.f;
    v[i].y = w[i] > d.above ? v[i].y * d.scale : 0.f;
  }
}

// Which of the eight elements of a block are kept, a bit each.
__device__ __forceinline__ uint32_t kept8(const Drop& d, uint64_t block, uint64_t call, uint64_t seed) {
  const uint4 r = philox(block, call, seed);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= (w[i] << 16 > d.above ? 1u << 2 * i : 0u) | (w[i] > d.above ? 2u << 2 * i : 0u);
  return m;
}

}  // namespace scan
