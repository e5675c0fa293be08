// What the warp-specialised tensor-core kernels of the prompt operators share:
// bounded waits, registers of warpgroups, descriptors and products in BF16.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace sage {
namespace tc {

constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait
// Some roles wait for all tiles of a unit of work, and a unit may have eight million: 2 s
// and 20 us for each (a tile takes 0.3 to 1.5 us, a few where values are cleared).
inline uint64_t wait_limit_ns(int64_t tiles) { return kWaitNs + static_cast<uint64_t>(tiles) * 20000u; }

// Barriers and the abort word of a CTA, in shared memory. A wait that runs out
// sets the device error word and the abort word, which ends every other wait.
struct Waits {
  uint32_t bar0;
  volatile int* abort_flag;  // null: a wait of the clean-up, which goes on after an abort
  int* dev_err;
  uint64_t limit;            // of a wait, in ns
  __device__ uint32_t bar(int i) const { return bar0 + 8u * static_cast<uint32_t>(i); }
  __device__ Waits draining() const { return Waits{bar0, nullptr, dev_err, limit}; }
};

__device__ __forceinline__ bool wait_bar(const Waits& w, uint32_t bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 127u) == 0) {
      if (w.abort_flag != nullptr && *w.abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > w.limit) {
        if (w.abort_flag != nullptr) *w.abort_flag = 1;
        atomicExch(w.dev_err, kDevErrTimeout);
        return false;
      }
    }
  }
}

// Every lane waits; the warp goes on only if all did.
__device__ __forceinline__ bool wait_bar_warp(const Waits& w, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_bar(w, bar, parity));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two BF16 in a word, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// Registers are those of a whole warpgroup.
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// One lane of the warp, chosen by the hardware.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred != 0;
}

// Descriptor of the operand `offset` bytes behind another (buffers lie below
// 256 KB: no carry out of the address field).
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t offset) { return base + (offset >> 4); }

// Shared-memory descriptor of an operand whose rows run along K (each 128
// bytes of 64 BF16 of M or N; 128-byte swizzle): 8 rows of K are 1024 bytes, the
// next 64 of M or N are `next` bytes on.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr, uint32_t next) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(next >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// Instruction descriptor of kind::f16 with BF16 operands, fp32 sums, M = 128.
// kMnB: B runs along N in shared memory (sw128_mn_desc).
template <int N, bool kMnB = false>
struct IdescBf16 {
  static constexpr uint32_t value = (1u << 4) | (1u << 7) | (1u << 10) | (kMnB ? 1u << 16 : 0u) |
                                    (static_cast<uint32_t>(N >> 3) << 17) | ((128u >> 4) << 24);
};

// Brings a box of a tensor into L2.
__device__ __forceinline__ void tma_prefetch_3d(const void* tmap, int32_t c0, int32_t c1, int32_t c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(tmap)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// D(tmem) (+)= A(tmem) * B(smem), 16-bit operands, fp32 sums, K = 16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 columns (as tmem_ld32, tmem_st32).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

}  // namespace tc
}  // namespace sage
