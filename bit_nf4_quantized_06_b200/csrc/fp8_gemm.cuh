// Tensor-core product of 8-bit rows with an 8-bit weight: parameters and
// device helpers. For files compiled without relocatable device code, under
// which ptxas ignores setmaxnreg.
#pragma once

#define QLORA_STANDALONE

#include <cuda_bf16.h>

#include "fp8_dev.cuh"
#include "fp8_launch.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace qlora {

// Waits. On timeout (two seconds), or when another role has given up, false; a
// timeout sets `code` in the device status word.
struct Fp8Abort {
  volatile int* flag;       // shared memory, one a CTA
  unsigned int* status;     // the library's device status word
};

// A token: whether the phase is over, without waiting for it.
//
// What stands between a barrier's phase and the work that waits for it counts
// in full here (a reduction block is 256 or 512 cycles of tensor core), and a
// wait of the usual form costs 100 to 200 cycles even where the phase is long
// over: the try's latency, its loop and the vote that makes the answer the
// same in every lane. So a role first takes a token, looks at it after other
// work, and waits only where it failed; and warps do not vote: a wait that
// gives up just goes on (the flag then ends every later wait at its first try,
// and results are void), so lanes need not agree.
__device__ __forceinline__ bool fp8_token(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, const Fp8Abort& a, unsigned code) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*a.flag) return false;
  }
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*a.flag) return false;
    if (globaltimer_ns() - t0 > QLORA_WAIT_LIMIT_NS) {
      atomicOr(a.status, code);
      *a.flag = 1;
      return false;
    }
  }
}

// For the one thread that issues MMAs: asks again at once, where a suspended
// wait takes its time to wake (pair kernel, 1% of the time).
__device__ __forceinline__ bool fp8_spin(uint32_t bar, uint32_t parity, const Fp8Abort& a, unsigned code) {
#pragma unroll 1
  for (int i = 0; i < 256; ++i)
    if (fp8_token(bar, parity)) return true;
  return fp8_wait(bar, parity, a, code);
}

// Instruction descriptor for kind::f8f6f4: A e4m3 or e5m2, B e4m3, fp32 D.
__device__ __forceinline__ uint32_t idesc_fp8(int m, int n, int a_format, bool b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(a_format) << 7) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_fp8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive once on the barrier at this offset in both CTAs of the pair when
// every MMA issued so far by this thread completes.
__device__ __forceinline__ void tc_commit_both(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void tc_mma_fp8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns: thread i gets lane i.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// acc[i] += t[2i, 2i+1] * s, in pairs
__device__ __forceinline__ void promote16(uint64_t* acc, const uint32_t (&t)[16], uint64_t s2) {
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = f2_fma(f2(__uint_as_float(t[2 * i]), __uint_as_float(t[2 * i + 1])), s2, acc[i]);
}

}  // namespace qlora
