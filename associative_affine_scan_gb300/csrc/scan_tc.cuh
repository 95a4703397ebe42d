// scan_tc.cuh -- the tensor-core (tcgen05), tensor-memory and tensor-copy (TMA)
// instructions that the attention kernels are written with, one wrapper each,
// and the layouts that tie them together.
//
// Operand tiles in shared memory are panels of 64 bf16 columns (128 bytes) by
// any number of rows, row pitch 128 bytes, the 16-byte pieces of a row permuted
// by the row number modulo 8 (the 128-byte swizzle that tensor copies write). A
// panel starts on 1024 bytes. The same tile serves two ways:
//   - K-major: rows are M or N, columns are the summed index. Eight rows are
//     1024 bytes apart; 16 columns further is 32 bytes further.
//   - MN-major: columns are M or N, rows are the summed index. Panels of 64
//     columns are `panel` bytes apart; 16 rows further is 2048 bytes further.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "scan_internal.h"

namespace scan {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ---- mbarriers -------------------------------------------------------------

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.shared::cta.b64 t, [%0];\n}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .b64 t;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n}" ::"r"(bar),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

constexpr uint64_t kWaitNs = 1000000000ull;  // every wait gives up after a second

// What a block's waits share: once one has expired the rest return at once and
// every role leaves its loop. The expiry is recorded in the workspace's status.
struct Stop {
  volatile uint32_t* flag;  // in shared memory
  WsHeader* hdr;
};

static __device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, const Stop& s) {
  const uint64_t t0 = now_ns();
  while (!bar_try(bar, parity)) {
    if (*s.flag) return false;
    if (now_ns() - t0 > kWaitNs) {
      *s.flag = 1;
      s.hdr->status = SCAN_ERR_TIMEOUT;
      return false;
    }
  }
  return true;
}
// False: some wait of this block expired, leave.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, const Stop& s) {
  if (bar_try(bar, parity)) return true;
  return bar_wait_slow(bar, parity, s);
}
// The same for a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const Stop& s) {
  return __all_sync(0xffffffffu, bar_wait(bar, parity, s));
}
// After an expired wait copies may still be in flight towards the block's
// shared memory: stay until they must have landed.
__device__ __forceinline__ void linger(const Stop& s) {
  if (!*s.flag) return;
  const uint64_t t0 = now_ns();
  while (now_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// ---- tensor copies ---------------------------------------------------------

__device__ __forceinline__ void copy_in_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                           int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void copy_out_4d(const CUtensorMap* map, uint32_t src, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
      "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void copy_out_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void copy_out_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Orders this thread's shared-memory writes before the asynchronous reads
// (tensor cores, tensor copies) that a later barrier arrival starts.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory ---------------------------------------------------------

__device__ __forceinline__ void tmem_alloc(uint32_t where, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(where), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this warp's 32 lanes; addr carries the warp's first lane in its
// upper half. Results may be used after ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ---- products --------------------------------------------------------------

constexpr uint32_t kPitch = 128;  // bytes of a panel row

// A bf16 x bf16 -> fp32 product of M x N, either operand MN-major.
__device__ __forceinline__ constexpr uint32_t product_desc(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N / 8) << 17) | ((uint32_t)(M / 16) << 24);
}
// An operand's descriptor: the upper word is the same for all (rows of eight 1024
// bytes apart, 128-byte swizzle); the lower word holds the tile's address and, for
// MN-major tiles, the distance of its panels. One thread issues every product, and
// its instructions are what bounds the issue, so a tile's lower word is made once
// and steps along the summed index add constants to it.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t kmajor(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mnmajor(uint32_t addr, uint32_t panel) {
  return (addr >> 4) | ((panel >> 4) << 16);
}

// The product warp runs as a whole, so that descriptors and addresses stay in
// uniform registers, which these instructions read; `lead` (one lane) issues.
__device__ __forceinline__ void mma_ss(bool lead, uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"((uint32_t)add), "r"(kDescHigh), "r"((uint32_t)lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(bool lead, uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(desc), "r"((uint32_t)add), "r"(kDescHigh), "r"((uint32_t)lead)
      : "memory");
}
// Arrives on `bar` when every product issued by this thread has finished.
__device__ __forceinline__ void mma_commit(bool lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
      "r"((uint32_t)lead)
      : "memory");
}

// d (+)= A B^T over K = 64 * panels columns; A and B K-major tiles (kmajor() of
// their addresses) whose panels are AP and BP bytes apart.
template <int K, uint32_t AP, uint32_t BP>
__device__ __forceinline__ void mma_kk(bool lead, uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
#pragma unroll
  for (int k = 0; k < K / 16; ++k)
    mma_ss(lead, d, a + (k / 4) * (AP >> 4) + (k % 4) * 2, b + (k / 4) * (BP >> 4) + (k % 4) * 2, desc, add || k > 0);
}
// d (+)= A B over K rows; A in tensor memory (two bf16 a column), B MN-major
// (mnmajor() of its address).
template <int K>
__device__ __forceinline__ void mma_tn(bool lead, uint32_t d, uint32_t a, uint32_t b, uint32_t desc, bool add) {
#pragma unroll
  for (int k = 0; k < K / 16; ++k) mma_ts(lead, d, a + k * 8, b + k * (2048 >> 4), desc, add || k > 0);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void st_global32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 2^x by the special-function unit (flushes results below 2^-126 to 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Pairs of fp32 in one operation.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 pair_of(const uint32_t* r) {
  return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// Where piece `piece` (16 bytes) of row `row` of a panel lies.
__device__ __forceinline__ uint32_t swizzled(uint32_t panel, int row, int piece) {
  return panel + row * kPitch + ((piece ^ (row & 7)) << 4);
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
}  // namespace tc

}  // namespace scan
