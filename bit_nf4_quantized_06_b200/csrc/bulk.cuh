// Untiled bulk copies into shared memory, and loads from there.
#pragma once

#include "ptx.cuh"

namespace qlora {

// Bulk copy global -> this CTA's shared memory (both 16-byte aligned, a
// multiple of 16 bytes), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t lds_u1(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Up to 32 stages that one thread (the filler) has bulk copies fill and a group
// of threads reads. Every thread of the group keeps one of these.
//
// A wait that gives up is one thread's: the copy may land just then for the
// others. So no thread leaves on its own answer, which would leave the others at
// the group's next barrier. It sets the ring's flag and goes on; every later
// wait on a copy that is not there ends at its first tries, the filler requests
// nothing more, and before the shared memory goes to another use it lets what it
// requested land.
struct BulkRing {
  uint32_t bars;         // the stages' barriers in shared memory, 8 bytes each; in front of them a word of bits and the flag
  uint32_t phases = 0;   // a bit a stage: the parity that its next wait looks for

  __device__ __forceinline__ explicit BulkRing(uint32_t memory) : bars(memory + 8) {}
  __device__ __forceinline__ uint32_t bar(int s) const { return bars + 8u * s; }
  __device__ __forceinline__ void init(int stages) const {   // one thread, a barrier of the group behind it
    asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(bars - 8), "r"(0) : "memory");
    for (int s = 0; s < stages; ++s) mbar_init(bar(s), 1);
    fence_mbar_init();
  }
  __device__ __forceinline__ bool given_up() const { return lds_u1(bars - 4) != 0; }
  __device__ __forceinline__ void give_up(unsigned code) const {
    atomicOr(&g_dev_status, code);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(bars - 4), "r"(1) : "memory");
  }
  // The filler, in front of copies of `bytes` in all. The bits turn with every
  // filling as `phases` does with every wait: where they differ, copies are
  // under way.
  __device__ __forceinline__ void expect(int s, uint32_t bytes) const {
    mbar_arrive_expect_tx(bar(s), bytes);
    asm volatile("red.shared.xor.b32 [%0], %1;" ::"r"(bars - 8), "r"(1u << s) : "memory");
  }
  // Bounded; on timeout sets `code` in the status word, and the flag. False if
  // the copies have not landed: what the stage holds is void.
  __device__ __forceinline__ bool wait(int s, uint64_t limit_ns = QLORA_WAIT_LIMIT_NS,
                                       unsigned code = QLORA_DEV_TIMEOUT_PRODUCER) {
    const uint32_t b = bar(s), parity = (phases >> s) & 1;
    bool ok = mbar_try_wait(b, parity);
    if (!ok) {
      const uint64_t t0 = globaltimer_ns();
      while (!(ok = mbar_try_wait(b, parity)) && !given_up())
        if (globaltimer_ns() - t0 > limit_ns) give_up(code);
    }
    if (ok) phases ^= 1u << s;
    return ok;
  }
  // The filler, last of all: nothing to do unless a wait gave up. Bounded; false
  // if copies are still under way.
  __device__ __forceinline__ bool drain(uint64_t limit_ns = QLORA_WAIT_LIMIT_NS) const {
    uint32_t left = lds_u1(bars - 8) ^ phases;
    if (left == 0) return true;
    const uint64_t t0 = globaltimer_ns();
    for (; left != 0; left &= left - 1) {
      const int s = __ffs(left) - 1;
      while (!mbar_try_wait(bar(s), (phases >> s) & 1))
        if (globaltimer_ns() - t0 > limit_ns) return false;
    }
    return true;
  }
};
constexpr int ring_words(int stages) { return stages + 1; }   // 8-byte words of shared memory

__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ void lds_f4(uint32_t addr, float* f) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]) : "r"(addr));
}

}  // namespace qlora
