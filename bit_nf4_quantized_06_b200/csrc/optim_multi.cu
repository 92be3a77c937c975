// AdamW over many tensors in one launch, states in 32 bits or in 8 (sm_100a).
//
// A stack's adapters are hundreds of tensors of 10^4 to 10^6 values: one
// launch each costs more than the update. The descriptors travel as the
// kernel's parameters (no copy, nothing left to keep alive, capturable), and
// the CTAs walk the chunks of all tensors as one list.
//
// 8 bits: m and sqrt(v) are e4m3 codes with one fp32 scale per 256 values of
// a tensor; a warp owns a block, eight values a lane, so that
// the block's maxima are one warp operation each. sqrt(v) rather than v: e4m3 spans
// 2^17.8 from its smallest code to its largest, which is 2^35 of v. A code of
// a value above zero is not allowed to become zero, else the next step would
// divide by eps alone. The step uses the new m and v in fp32, so rounding
// them to 8 bits acts on later steps only.
//
// The states are defined operation by operation (the header has the list), so
// that a state after any number of steps is one set of bits: a value that a
// last bit moved over a rounding border would be a whole code away, and as its
// block's next largest value would move the scale by some per cent. With m in
// one fused operation 3 of 4 runs of four steps over 160 million values ended
// with such a block. amax / 448 and 448 / amax are products with a
// reciprocal, as torch's operators on a tensor and a number are on the GPU.
//
// Bound by HBM: 30 bytes a value (32 bits, with the bf16 copy) or 18.1 (8
// bits). A CTA takes chunks of eight blocks, a block a warp, through a ring of
// stages in shared memory: one stage holds a chunk's master values, gradients
// and states, filled by four bulk copies that are requested several chunks
// ahead. Measured, 8 bits, 160 million values in 448 tensors: 450 us, 6.4 TB/s,
// in runs of hundreds of steps, at the board's power limit, 475 to 500
// (loads to registers kept 61 KB in flight on an SM, 573 us; a ring a warp, of
// 256-byte copies, was bound by the copies' number, 816 us); 32 bits, 134
// million values: 688 us, 5.9 TB/s.
#include <algorithm>
#include <cmath>
#include <vector>

#include <cuda_bf16.h>

#include "../../include/qlora.h"
#include "adamw_math.cuh"
#include "bulk.cuh"
#include "fp8_dev.cuh"
#include "host.h"
#include "ptx.cuh"

namespace qlora {
namespace {

constexpr int kStateBlock = QLORA_ADAMW_STATE_BLOCK;
constexpr int kThreads = 256;
constexpr int kChunk = kThreads / 32 * kStateBlock;   // values of a chunk
constexpr float kLeastRoot = 1.0f / 512.0f;   // the smallest e4m3 code above zero

struct MultiTensor {
  float* master;
  __nv_bfloat16* param;
  const float* grad;
  void* m;
  void* v;
  float* m_scales;
  float* v_scales;
  int64_t n;
};

// Up to CAP tensors: two capacities, so that a few tensors do not pay for the
// copy of a 32 KB parameter block at launch.
template <int CAP>
struct Multi {
  MultiTensor t[CAP];
  int32_t first[CAP];       // the tensor's first chunk in the list of all; bit 31: wide accesses allowed
  int32_t count;
  int32_t chunks;
  AdamwHyper hp;
};
constexpr int kCapSmall = 24, kCapLarge = 470;
static_assert(sizeof(Multi<kCapLarge>) <= 32764, "kernel parameter block");

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float lo_of(uint64_t v) {
  uint32_t a, b;
  f2_split(v, a, b);
  return __uint_as_float(a);
}
__device__ __forceinline__ float hi_of(uint64_t v) {
  uint32_t a, b;
  f2_split(v, a, b);
  return __uint_as_float(b);
}

// Constants of the 8-bit step; the update's in pairs.
struct Hyper2 {
  float beta1, gain1, beta2, gain2, one;
  uint64_t decay, neg_step, inv_sqrt_bc2, eps;
};
__device__ __forceinline__ Hyper2 hyper2(const AdamwHyper& a) {
  auto two = [](float v) { return f2(v, v); };
  return Hyper2{a.beta1,      1.0f - a.beta1,    a.beta2,             1.0f - a.beta2, a.one,
                two(a.decay), two(-a.step_size), two(a.inv_sqrt_bc2), two(a.eps)};
}

// a x + b y in pairs, each product and the sum rounded by itself. The assembler
// joins a packed product and a packed sum into one fused operation, `.rn` or
// not; a sum as x * one + y, with a one that it does not know, it leaves as it is.
__device__ __forceinline__ uint64_t sum_apart(float a, uint64_t x, float b, uint64_t y, float one) {
  return f2_fma(f2_mul(f2(a, a), x), f2(one, one), f2_mul(f2(b, b), y));
}

// The largest of a warp's values, NaN aside.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}

// Where a block's values lie in a stage; p == 0: nowhere.
struct Stage {
  uint32_t p, g, m, v;
};

// A lane's eight values of a block: 4 lane + (0..3) and 128 + 4 lane + (0..3),
// so that every access of a warp is one contiguous piece.
__device__ __forceinline__ int value_of(int lane, int j) { return (j >> 2) * 128 + 4 * lane + (j & 3); }

// The 8-bit step of the block at i0 (`src`: its stage, or 0 for plain
// accesses; `read` is called once its values are in registers, and says whether
// they may be used), in packed pairs. The states' operations are rounded one by
// one; the rounded square root takes 20 to 30 us more of 160 million values than
// the hardware's approximate one, with which states were not reproducible. The
// update's reciprocal, which no state depends on, is the hardware's, off by one
// step of fp32 at most: with a rounded quotient too this kernel was bound by
// issue (83 instructions a value, 654 us).
template <typename Read>
__device__ __forceinline__ void step8(const MultiTensor& t, int64_t i0, int lane, const Stage& src, const Hyper2& hp,
                                      Read read) {
  const int64_t blk = i0 / kStateBlock;
  const int left = static_cast<int>(min(static_cast<int64_t>(kStateBlock), t.n - i0));
  const float ms = t.m_scales[blk], vs = t.v_scales[blk];
  uint8_t* mc = static_cast<uint8_t*>(t.m) + i0;
  uint8_t* vc = static_cast<uint8_t*>(t.v) + i0;
  float p[8], g[8];
  uint2 mq, vq;
  if (src.p != 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lds_f4(src.p + 512 * h + 16 * lane, p + 4 * h);
      lds_f4(src.g + 512 * h + 16 * lane, g + 4 * h);
    }
    mq = make_uint2(lds_u1(src.m + 4 * lane), lds_u1(src.m + 128 + 4 * lane));
    vq = make_uint2(lds_u1(src.v + 4 * lane), lds_u1(src.v + 128 + 4 * lane));
  } else {
    uint32_t mb[8], vb[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = value_of(lane, j);
      const bool ok = c < left;
      p[j] = ok ? t.master[i0 + c] : 0.0f;
      g[j] = ok ? t.grad[i0 + c] : 0.0f;
      mb[j] = ok ? mc[c] : 0u;
      vb[j] = ok ? vc[c] : 0u;
    }
    mq = make_uint2(mb[0] | mb[1] << 8 | mb[2] << 16 | mb[3] << 24, mb[4] | mb[5] << 8 | mb[6] << 16 | mb[7] << 24);
    vq = make_uint2(vb[0] | vb[1] << 8 | vb[2] << 16 | vb[3] << 24, vb[4] | vb[5] << 8 | vb[6] << 16 | vb[7] << 24);
  }
  if (!read()) return;
  const uint64_t ms2 = f2(ms, ms), vs2 = f2(vs, vs);
  float m[8], r[8];
  float am = 0.0f, av = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint32_t sh = 8 * (j & 3);
    const float2 mm = fp8_unpack2<kE4M3>((j < 4 ? mq.x : mq.y) >> sh);
    const float2 rr = fp8_unpack2<kE4M3>((j < 4 ? vq.x : vq.y) >> sh);
    const uint64_t g2 = f2(g[j], g[j + 1]);
    const uint64_t m2 = sum_apart(hp.beta1, f2_mul(f2(mm.x, mm.y), ms2), hp.gain1, g2, hp.one);
    const uint64_t r2 = f2_mul(f2(rr.x, rr.y), vs2);
    const uint64_t v2 = sum_apart(hp.beta2, f2_mul(r2, r2), hp.gain2, f2_mul(g2, g2), hp.one);
    r[j] = __fsqrt_rn(lo_of(v2));
    r[j + 1] = __fsqrt_rn(hi_of(v2));
    const uint64_t d2 = f2_fma(f2(r[j], r[j + 1]), hp.inv_sqrt_bc2, hp.eps);
    const uint64_t q2 = f2_mul(m2, f2(rcp_approx(lo_of(d2)), rcp_approx(hi_of(d2))));
    const uint64_t p2 = f2_fma(hp.neg_step, q2, f2_mul(f2(p[j], p[j + 1]), hp.decay));
    p[j] = lo_of(p2);
    p[j + 1] = hi_of(p2);
    m[j] = lo_of(m2);
    m[j + 1] = hi_of(m2);
    am = fmaxf(am, fmaxf(fabsf(m[j]), fabsf(m[j + 1])));
    av = fmaxf(av, fmaxf(r[j], r[j + 1]));
  }
  am = warp_max(am);
  av = warp_max(av);
  if (fmaxf(am, av) > FLT_MAX) {               // the same for the whole warp: infinities become NaN
    am = av = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      am = fmaxf(am, fp8_mag(m[j]));
      av = fmaxf(av, fp8_mag(r[j]));
      m[j] += m[j] - m[j];
      r[j] += r[j] - r[j];
    }
    am = warp_max(am);
    av = warp_max(av);
  }
  constexpr float F = 448.0f;
  am = fmaxf(am, kFp8Least);
  av = fmaxf(av, kFp8Least);
  const float im = F * __frcp_rn(am), iv = F * __frcp_rn(av);
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const uint64_t cm = f2_mul(f2(m[j], m[j + 1]), f2(im, im)), cr = f2_mul(f2(r[j], r[j + 1]), f2(iv, iv));
    m[j] = lo_of(cm);
    m[j + 1] = hi_of(cm);
    r[j] = r[j] > 0.0f ? fmaxf(lo_of(cr), kLeastRoot) : lo_of(cr);
    r[j + 1] = r[j + 1] > 0.0f ? fmaxf(hi_of(cr), kLeastRoot) : hi_of(cr);
  }
  mq = make_uint2(fp8_pack4<kE4M3>(m[0], m[1], m[2], m[3]), fp8_pack4<kE4M3>(m[4], m[5], m[6], m[7]));
  vq = make_uint2(fp8_pack4<kE4M3>(r[0], r[1], r[2], r[3]), fp8_pack4<kE4M3>(r[4], r[5], r[6], r[7]));
  if (lane < 2) {
    float* scale = lane == 0 ? t.m_scales : t.v_scales;
    scale[blk] = (lane == 0 ? am : av) * (1.0f / F);
  }
  if (src.p != 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = i0 + 128 * h + 4 * lane;
      *reinterpret_cast<float4*>(t.master + at) = make_float4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]);
      reinterpret_cast<uint32_t*>(mc)[32 * h + lane] = h == 0 ? mq.x : mq.y;
      reinterpret_cast<uint32_t*>(vc)[32 * h + lane] = h == 0 ? vq.x : vq.y;
      if (t.param != nullptr)
        *reinterpret_cast<uint2*>(t.param + at) =
            make_uint2(pack_bf16x2(p[4 * h], p[4 * h + 1]), pack_bf16x2(p[4 * h + 2], p[4 * h + 3]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = value_of(lane, j);
      if (c >= left) continue;
      t.master[i0 + c] = p[j];
      mc[c] = static_cast<uint8_t>((j < 4 ? mq.x : mq.y) >> (8 * (j & 3)));
      vc[c] = static_cast<uint8_t>((j < 4 ? vq.x : vq.y) >> (8 * (j & 3)));
      if (t.param != nullptr) t.param[i0 + c] = __float2bfloat16_rn(p[j]);
    }
  }
}

// The same with fp32 states, in the arithmetic of qlora_adamw_step.
template <typename Read>
__device__ __forceinline__ void step32(const MultiTensor& t, int64_t i0, int lane, const Stage& src,
                                       const AdamwHyper& hp, Read read) {
  const int left = static_cast<int>(min(static_cast<int64_t>(kStateBlock), t.n - i0));
  float* ms = static_cast<float*>(t.m) + i0;
  float* vs = static_cast<float*>(t.v) + i0;
  float p[8], g[8], m[8], v[8], root;
  if (src.p != 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lds_f4(src.p + 512 * h + 16 * lane, p + 4 * h);
      lds_f4(src.g + 512 * h + 16 * lane, g + 4 * h);
      lds_f4(src.m + 512 * h + 16 * lane, m + 4 * h);
      lds_f4(src.v + 512 * h + 16 * lane, v + 4 * h);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = value_of(lane, j);
      const bool ok = c < left;
      p[j] = ok ? t.master[i0 + c] : 0.0f;
      g[j] = ok ? t.grad[i0 + c] : 0.0f;
      m[j] = ok ? ms[c] : 0.0f;
      v[j] = ok ? vs[c] : 0.0f;
    }
  }
  if (!read()) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) p[j] = adamw_update(p[j], g[j], m[j], v[j], root, hp);
  if (src.p != 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 128 * h + 4 * lane;
      *reinterpret_cast<float4*>(t.master + i0 + c) = make_float4(p[4 * h], p[4 * h + 1], p[4 * h + 2], p[4 * h + 3]);
      *reinterpret_cast<float4*>(ms + c) = make_float4(m[4 * h], m[4 * h + 1], m[4 * h + 2], m[4 * h + 3]);
      *reinterpret_cast<float4*>(vs + c) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
      if (t.param != nullptr)
        *reinterpret_cast<uint2*>(t.param + i0 + c) =
            make_uint2(pack_bf16x2(p[4 * h], p[4 * h + 1]), pack_bf16x2(p[4 * h + 2], p[4 * h + 3]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = value_of(lane, j);
      if (c >= left) continue;
      t.master[i0 + c] = p[j];
      ms[c] = m[j];
      vs[c] = v[j];
      if (t.param != nullptr) t.param[i0 + c] = __float2bfloat16_rn(p[j]);
    }
  }
}

constexpr int kStages = 2;
constexpr int stage_bytes(bool b8) { return kChunk * (b8 ? 10 : 16); }

template <int CAP, bool BITS8>
__global__ void __launch_bounds__(kThreads, 3) k_adamw_multi(const __grid_constant__ Multi<CAP> a) {
  extern __shared__ __align__(128) uint8_t s_ring[];
  __shared__ __align__(8) uint64_t s_bar[ring_words(kStages)];
  constexpr uint32_t W = BITS8 ? 1 : 4;          // bytes of a state
  constexpr uint32_t STAGE = stage_bytes(BITS8);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t base = smem_u32(s_ring);
  BulkRing ring(smem_u32(s_bar));
  if (threadIdx.x == 0) ring.init(kStages);
  __syncthreads();
  grid_dependency_wait();
  grid_dependency_trigger();
  const Hyper2 hp2 = hyper2(a.hp);
  auto first = [&](int i) { return a.first[i] & 0x7FFFFFFF; };
  const int stride = gridDim.x;
  // cursors over this CTA's chunks: the one at work and the one to request
  struct Cursor {
    int chunk, t;
  };
  auto settle = [&](Cursor& c) {     // the last tensor whose first chunk is not past c.chunk
    while (c.t + 1 < a.count && first(c.t + 1) <= c.chunk) ++c.t;
  };
  auto whole = [&](const Cursor& c) {   // a whole chunk of a tensor that takes wide accesses
    return a.first[c.t] < 0 && static_cast<int64_t>(c.chunk - first(c.t) + 1) * kChunk <= a.t[c.t].n;
  };
  auto request = [&](const Cursor& c, int s) {   // one thread
    if (c.chunk >= a.chunks || !whole(c) || ring.given_up()) return;
    const MultiTensor& t = a.t[c.t];
    const int64_t i0 = static_cast<int64_t>(c.chunk - first(c.t)) * kChunk;
    const uint32_t dst = base + s * STAGE, bar = ring.bar(s);
    ring.expect(s, STAGE);
    bulk_load(dst, t.master + i0, kChunk * 4, bar);
    bulk_load(dst + kChunk * 4, t.grad + i0, kChunk * 4, bar);
    bulk_load(dst + kChunk * 8, static_cast<const uint8_t*>(t.m) + i0 * W, kChunk * W, bar);
    bulk_load(dst + kChunk * (8 + W), static_cast<const uint8_t*>(t.v) + i0 * W, kChunk * W, bar);
  };
  Cursor cur{static_cast<int>(blockIdx.x), 0}, ahead{};
  {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first(mid) <= cur.chunk)
        lo = mid;
      else
        hi = mid - 1;
    }
    cur.t = lo;
  }
  ahead = cur;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      settle(ahead);
      request(ahead, s);
      ahead.chunk += stride;   // at most 2^30 chunks: no overflow
    }
  }
  int s = 0;
  for (; cur.chunk < a.chunks; cur.chunk += stride) {
    settle(cur);
    const MultiTensor& t = a.t[cur.t];
    const int64_t i0 = static_cast<int64_t>(cur.chunk - first(cur.t)) * kChunk + warp * kStateBlock;
    Stage src{0, 0, 0, 0};
    bool ok = true;
    if (whole(cur)) {
      ok = ring.wait(s);
      const uint32_t at = base + s * STAGE;
      src = Stage{at + warp * 1024, at + kChunk * 4 + warp * 1024, at + kChunk * 8 + warp * (kStateBlock * W),
                  at + kChunk * (8 + W) + warp * (kStateBlock * W)};
    }
    auto read = [&]() {
      __syncthreads();         // every warp has read its part of the stage
      if (threadIdx.x == 0) {
        settle(ahead);
        request(ahead, s);
        ahead.chunk += stride;
      }
      return __all_sync(0xFFFFFFFFu, ok);   // a warp whose copies did not land in time writes nothing
    };
    if (i0 >= t.n)
      read();
    else if (BITS8)
      step8(t, i0, lane, src, hp2, read);
    else
      step32(t, i0, lane, src, a.hp, read);
    s = s + 1 == kStages ? 0 : s + 1;
  }
  if (threadIdx.x == 0) ring.drain();
}

using host::aligned;
using host::cdiv;

template <int CAP, bool BITS8>
int launch_multi(const qlora_adamw_tensor_t* t, const int* index, int count, const AdamwHyper& hp, int sms,
                 cudaStream_t st) {
  Multi<CAP> a;
  a.count = count;
  a.hp = hp;
  int64_t chunks = 0;
  for (int i = 0; i < count; ++i) {
    const qlora_adamw_tensor_t& s = t[index[i]];
    a.t[i] = MultiTensor{s.master, static_cast<__nv_bfloat16*>(s.param_bf16), s.grad, s.m, s.v,
                         s.m_scales, s.v_scales, s.n};
    const bool vec = aligned(s.master, 16) && aligned(s.grad, 16) && aligned(s.m, 16) && aligned(s.v, 16) &&
                     aligned(s.param_bf16, 8);
    a.first[i] = static_cast<int32_t>(chunks) | (vec ? static_cast<int32_t>(0x80000000u) : 0);
    chunks += cdiv(s.n, kChunk);
  }
  a.chunks = static_cast<int32_t>(chunks);
  // as many CTAs as the rings leave room for on an SM
  const int64_t resident = static_cast<int64_t>(sms) * 3;
  const int grid = static_cast<int>(std::min<int64_t>(chunks, resident));
  return host::launch_pdl(k_adamw_multi<CAP, BITS8>, dim3(grid), dim3(kThreads), kStages * stage_bytes(BITS8), st, 1, a);
}

// Whether two of the ranges [at(i), at(i) + bytes(i)) of the listed tensors overlap.
template <typename At, typename Bytes>
bool overlap(const std::vector<int>& live, At at, Bytes bytes) {
  bool ascending = true;
  for (size_t i = 1; ascending && i < live.size(); ++i)
    ascending = at(live[i - 1]) + bytes(live[i - 1]) <= at(live[i]);
  if (ascending) return false;     // the usual case: laid out one after the other
  std::vector<std::pair<uintptr_t, uintptr_t>> r;
  r.reserve(live.size());
  for (int i : live) r.emplace_back(at(i), at(i) + bytes(i));
  std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].second) return true;
  return false;
}

}  // namespace

cudaError_t set_adamw_attributes() {
  const auto a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(k_adamw_multi<kCapSmall, true>, a, kStages * stage_bytes(true));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_adamw_multi<kCapLarge, true>, a, kStages * stage_bytes(true));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_adamw_multi<kCapSmall, false>, a, kStages * stage_bytes(false));
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_adamw_multi<kCapLarge, false>, a, kStages * stage_bytes(false));
  return e;
}

}  // namespace qlora

using namespace qlora;

extern "C" qlora_status_t qlora_adamw_multi(const qlora_adamw_tensor_t* tensors, int64_t count, int32_t state_bits,
                                            const qlora_adamw_t* hp, void* stream) {
  if (hp == nullptr || count < 0 || (count > 0 && tensors == nullptr) || (state_bits != 8 && state_bits != 32))
    return QLORA_ERR_INVALID_ARG;
  if (count > (int64_t(1) << 24)) return QLORA_ERR_SHAPE;
  if (hp->step < 1 || !(hp->lr >= 0.0f) || !std::isfinite(hp->lr) || !(hp->beta1 >= 0.0f && hp->beta1 < 1.0f) ||
      !(hp->beta2 >= 0.0f && hp->beta2 < 1.0f) || !(hp->eps > 0.0f) || !std::isfinite(hp->eps) ||
      !std::isfinite(hp->weight_decay))
    return QLORA_ERR_INVALID_ARG;
  const bool b8 = state_bits == 8;
  try {
    std::vector<int> live;
    live.reserve(static_cast<size_t>(count));
    for (int64_t i = 0; i < count; ++i) {
      const qlora_adamw_tensor_t& t = tensors[i];
      if (t.n < 0 || t.n > (int64_t(1) << 38)) return QLORA_ERR_SHAPE;
      if (t.n == 0) continue;
      if (t.master == nullptr || t.grad == nullptr || t.m == nullptr || t.v == nullptr ||
          (b8 && (t.m_scales == nullptr || t.v_scales == nullptr)))
        return QLORA_ERR_INVALID_ARG;
      if (!aligned(t.master, 4) || !aligned(t.grad, 4) || !aligned(t.param_bf16, 2) ||
          (b8 ? !aligned(t.m_scales, 4) || !aligned(t.v_scales, 4) : !aligned(t.m, 4) || !aligned(t.v, 4)))
        return QLORA_ERR_ALIGNMENT;
      live.push_back(static_cast<int>(i));
    }
    if (live.empty()) return QLORA_OK;
    const size_t w = b8 ? 1 : 4;
    auto addr = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
    auto n = [&](int i) { return static_cast<uintptr_t>(tensors[i].n); };
    if (overlap(live, [&](int i) { return addr(tensors[i].master); }, [&](int i) { return 4 * n(i); }) ||
        overlap(live, [&](int i) { return addr(tensors[i].m); }, [&](int i) { return w * n(i); }) ||
        overlap(live, [&](int i) { return addr(tensors[i].v); }, [&](int i) { return w * n(i); }))
      return QLORA_ERR_INVALID_ARG;
    int sms = 0;
    qlora_status_t s = static_cast<qlora_status_t>(check_current_device(OpFamily::kAdamw, &sms));
    if (s != QLORA_OK) return s;
    // step constants in double, rounded once, as qlora_adamw_step has them
    AdamwHyper h{};
    h.beta1 = hp->beta1;
    h.beta2 = hp->beta2;
    h.eps = hp->eps;
    h.one = 1.0f;
    h.decay = static_cast<float>(1.0 - static_cast<double>(hp->lr) * hp->weight_decay);
    h.step_size = static_cast<float>(hp->lr / (1.0 - std::pow(static_cast<double>(hp->beta1), hp->step)));
    h.inv_sqrt_bc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(static_cast<double>(hp->beta2), hp->step)));
    if (b8 && h.eps < FLT_MIN) {
      // rcp_approx takes a denominator below the normal numbers for zero, and 0 / eps would be
      // NaN: the denominator and the step size both times 2^30, which rounds nothing (roots are
      // at most 2^64 and their correction below 2^13)
      constexpr float kUp = 1073741824.0f;
      h.eps *= kUp;
      h.inv_sqrt_bc2 *= kUp;
      h.step_size *= kUp;
      if (!std::isfinite(h.step_size)) return QLORA_ERR_INVALID_ARG;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // as many tensors a launch as its parameter block and 31-bit chunk numbers hold
    for (size_t at = 0; at < live.size();) {
      size_t to = at;
      int64_t chunks = 0;
      while (to < live.size() && to - at < kCapLarge) {
        const int64_t more = cdiv(tensors[live[to]].n, kChunk);
        if (to > at && chunks + more > (int64_t(1) << 30)) break;
        chunks += more;
        ++to;
      }
      const int k = static_cast<int>(to - at);
      const int rc = k <= kCapSmall ? (b8 ? launch_multi<kCapSmall, true>(tensors, &live[at], k, h, sms, st)
                                          : launch_multi<kCapSmall, false>(tensors, &live[at], k, h, sms, st))
                                    : (b8 ? launch_multi<kCapLarge, true>(tensors, &live[at], k, h, sms, st)
                                          : launch_multi<kCapLarge, false>(tensors, &live[at], k, h, sms, st));
      if (rc != QLORA_OK) return static_cast<qlora_status_t>(rc);
      at = to;
    }
  } catch (...) {   // only the host vectors' memory can fail
    return QLORA_ERR_CUDA;
  }
  return QLORA_OK;
}
