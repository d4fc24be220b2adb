// What the products with packed weights share: fp16 tensor-core products and shared-memory access.
#pragma once

#include "nvfp4.cuh"

namespace lhcal {

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a sum that starts at zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void sts_float(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void sts128(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Asynchronous copies into shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_word_async(uint32_t dst, const uint8_t* src, int bytes = 4) {  // zeros after `bytes`
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Barriers in shared memory that copies and products arrive at.
#ifdef LHCAL_IMPATIENT  // a build for tests, whose waits give up after one look
#define LHCAL_POLL "mbarrier.test_wait"
constexpr bool kImpatient = true;
#else
#define LHCAL_POLL "mbarrier.try_wait"
constexpr bool kImpatient = false;
#endif
constexpr int kWaitLimit = kImpatient ? 0 : 1 << 20;  // polls of a barrier, after which the CTA's results become NaN
constexpr int kDrainLimit = 1 << 20;  // the same of copies in flight, before a CTA that gave up ends
constexpr int kNan = 0x7fffffff;      // fp32
__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_poll(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t" LHCAL_POLL ".parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(bar), "r"(parity) : "memory");
  return done != 0;
}
// False if the limit is reached, here or elsewhere in the CTA: `failed` is then NaN's bits for good, else 0.
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, volatile int* failed) {
  if (barrier_poll(bar, parity)) return true;
  for (int i = 0; i < kWaitLimit; ++i) {
    if (barrier_poll(bar, parity)) return true;
    if (*failed) return false;
  }
  *failed = kNan;
  return false;
}
// The largest magnitude of bf16 pairs so far, as two 16-bit numbers.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t top, uint32_t u) { return __vmaxu2(top, u & 0x7fff7fffu); }
// Two bf16 values times a power of two (a bf16 pair), as an fp16 pair.
__device__ __forceinline__ uint32_t bf16x2_to_f16(uint32_t u, uint32_t up) {
  uint32_t v, r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(u), "r"(up));
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(__uint_as_float(v & 0xffff0000u)), "f"(__uint_as_float(v << 16)));
  return r;
}
// The power of two that brings the larger of two bf16 magnitudes to [2^14, 2^15), as a bf16 pair, and
// its inverse: 2^(141 - E) moves its exponent E to 14. Kept below 2^127, so that its inverse is a normal number.
__device__ __forceinline__ void fp16_range(uint32_t top, uint32_t& up, float& down) {
  const int e = min(141 - static_cast<int>(max(top >> 23, top << 16 >> 23)), 126);
  up = static_cast<uint32_t>(e + 127) * 0x800080u;
  down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

}  // namespace lhcal
