// RMS norm with the residual's addition, and its gradients (sm_100a).
//
//   h = bf16(x + res);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gamma
//   dx = rstd (dy g - h rstd^2 mean(dy g h)) + dres;  dgamma = sum_rows dy h rstd
//
// Both are streams over the rows, bound by HBM bandwidth (7 bytes a value
// forward with a residual and 8-bit output, 8 backward with a residual), so a
// row is read once and stays in registers between its statistics and its
// output. A group of T threads owns a row; warps own chunks of 256 columns.
// Measured: forward, 4096 rows of 8192, residual, 8-bit output 41 us (5.8 TB/s);
// backward, 4096 rows of 4096, residual 27 us (5.0 TB/s, the last sum over CTAs
// included).
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "bulk.cuh"
#include "fp8_dev.cuh"
#include "fp8_launch.h"
#include "host.h"
#include "ptx.cuh"
#include "../../include/qlora.h"

namespace qlora {
namespace {

constexpr int kChunk = 256;  // columns of one warp and step: 8 a lane

struct NormFwd {
  const __nv_bfloat16* x;
  const __nv_bfloat16* res;    // null: h = x
  const __nv_bfloat16* gamma;
  __nv_bfloat16* h;            // null without a residual
  __nv_bfloat16* y;            // bf16 output
  uint8_t* codes;              // 8-bit output
  float* scales;
  float* rstd;                 // may be null
  int64_t rows, d, ld;         // ld: bytes from row to row of codes
  int64_t nblk;                // scales per row
  float eps, inv_d;
};

struct NormBwd {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* h;
  const __nv_bfloat16* gamma;
  const float* rstd;
  const __nv_bfloat16* dres;   // may be null
  __nv_bfloat16* dx;
  float* part;                 // [gridDim.x][d], null without dgamma
  int64_t rows, d;
  float inv_d;
  int stages;                  // bulk stages; 0: plain loads
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a * b + c of the halves (lo or hi) of two bf16 pairs: the product is exact,
// one rounding to fp32.
__device__ __forceinline__ float fma_lo(uint32_t a, uint32_t b, float c) {
  float d;
  asm("{ .reg .b16 al, ah, bl, bh; mov.b32 {al, ah}, %1; mov.b32 {bl, bh}, %2; fma.rn.f32.bf16 %0, al, bl, %3; }"
      : "=f"(d)
      : "r"(a), "r"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float fma_hi(uint32_t a, uint32_t b, float c) {
  float d;
  asm("{ .reg .b16 al, ah, bl, bh; mov.b32 {al, ah}, %1; mov.b32 {bl, bh}, %2; fma.rn.f32.bf16 %0, ah, bh, %3; }"
      : "=f"(d)
      : "r"(a), "r"(b), "f"(c));
  return d;
}

// bf16(a + b) of two pairs, the sum rounded once. (Rounding it to fp32 first
// gives the same: a sum that fp32 does not hold is far from a tie of bf16.)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A lane's 8 values of a chunk. VEC: columns c0 + 8 lane + j, one 16-byte
// access (d % 8 == 0); else columns c0 + lane + 32 j, so that 2-byte accesses
// of a warp fall into one line. Packed as bf16 pairs (2i, 2i + 1).
template <bool VEC>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int c0, int lane, int d) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (VEC) {
    const int c = c0 + 8 * lane;
    if (c < d) v = *reinterpret_cast<const uint4*>(row + c);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + lane + 32 * j;
      w[j] = c < d ? p[c] : 0u;
    }
    v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return v;
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c0, int lane, int d, uint4 v) {
  if (VEC) {
    const int c = c0 + 8 * lane;
    if (c < d) *reinterpret_cast<uint4*>(row + c) = v;
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(row);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + lane + 32 * j;
      if (c < d) p[c] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf_lo(w[i]);
    f[2 * i + 1] = bf_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Quantize and store a lane's 8 values of a chunk: the chunk's two blocks of
// 128 columns are lanes 0-15 and 16-31 (VEC) or values 0-3 and 4-7.
template <bool VEC, int FMT>
__device__ __forceinline__ void store_fp8(uint8_t* row, float* scales, int c0, int lane, int d, float (&f)[8]) {
  constexpr float F = fp8_top<FMT>();
  constexpr int NB = VEC ? 1 : 2;              // blocks that a lane has values of
  constexpr int REACH = VEC ? 8 : 16;          // lanes that share a block: 16 or 32
  float a[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    a[b] = 0.0f;
#pragma unroll
    for (int j = 0; j < 8 / NB; ++j) a[b] = fmaxf(a[b], fabsf(f[8 / NB * b + j]));
#pragma unroll
    for (int o = REACH; o > 0; o >>= 1) a[b] = fmaxf(a[b], __shfl_xor_sync(0xFFFFFFFFu, a[b], o));
  }
  if (__any_sync(0xFFFFFFFFu, a[0] > FLT_MAX || a[NB - 1] > FLT_MAX)) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      a[b] = 0.0f;
#pragma unroll
      for (int j = 0; j < 8 / NB; ++j) {
        float& v = f[8 / NB * b + j];
        a[b] = fmaxf(a[b], fp8_mag(v));
        v += v - v;                            // an infinity becomes NaN
      }
#pragma unroll
      for (int o = REACH; o > 0; o >>= 1) a[b] = fmaxf(a[b], __shfl_xor_sync(0xFFFFFFFFu, a[b], o));
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) a[b] = fmaxf(a[b], kFp8Least);
  if (VEC) {
    const float inv = F / a[0];
    const int c = c0 + 8 * lane;
    if (c < d) {
      uint2 q;
      q.x = fp8_pack4<FMT>(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
      q.y = fp8_pack4<FMT>(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
      *reinterpret_cast<uint2*>(row + c) = q;
      if ((lane & 15) == 0) scales[c >> 7] = a[0] / F;
    }
  } else {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float inv = F / a[b];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = c0 + lane + 32 * (4 * b + j);
        const float s = f[4 * b + j] * inv;
        if (c < d) row[c] = static_cast<uint8_t>(fp8_pack2<FMT>(s, s));
      }
      if (lane == 0 && c0 + 128 * b < d) scales[(c0 >> 7) + b] = a[b] / F;
    }
  }
}

// Barrier of the threads of a row group (threadIdx.y < 15, whole warps).
__device__ __forceinline__ void group_sync(int warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(warps * 32) : "memory");
}

// Sum over the T threads of a row group; `red` has as many floats as a group
// has warps. OWN: the group meets at a barrier of its own, else the whole CTA.
template <bool OWN>
__device__ __forceinline__ float group_sum(float v, float* red, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[w] = v;
  if (OWN)
    group_sync(warps);
  else
    __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.0f);
}

constexpr int kBwdMaxStages = 8;
constexpr size_t kBwdMaxSmem = 220 * 1024;

enum NormOut : int { kOutBf16 = 0, kOutE4M3 = 1, kOutE5M2 = 2 };

// NV chunks a warp, kept in registers; NV == 0: any width, h is read again
// for the output (rows of over 16384 values).
// NORM false: the rows are only quantized (y = x).
template <int NV, bool VEC, int OUT, bool NORM>
__global__ void __launch_bounds__(NV == 0 ? 1024 : 512) k_rows_fwd(NormFwd p) {
  __shared__ float s_red[32 * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = row < p.rows;
  const int d = live ? static_cast<int>(p.d) : 0;     // an idle group reads and writes nothing
  const int width = static_cast<int>(p.d);
  const __nv_bfloat16* x = p.x + row * p.d;
  const __nv_bfloat16* res = p.res + row * p.d;
  constexpr int KEEP = NV > 0 ? NV : 1;
  const int step = warps * kChunk;
  const int nstep = NV > 0 ? NV : (width + step - 1) / step;
  uint4 keep[KEEP];
  grid_dependency_wait();
  grid_dependency_trigger();

  // on bf16 pairs as they are: this kernel is as much bound by issue as by HBM
  auto add = [&](uint4 a, uint4 b) {
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
  };
  float sum[2] = {0.0f, 0.0f};
  auto square = [&](uint4 t) {
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sum[0] = fma_lo(w[i], w[i], sum[0]);
      sum[1] = fma_hi(w[i], w[i], sum[1]);
    }
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) keep[v] = load8<VEC>(x, v * step + warp * kChunk, lane, d);
    if (NORM && p.res != nullptr) {
      uint4 other[KEEP];
#pragma unroll
      for (int v = 0; v < NV; ++v) other[v] = load8<VEC>(res, v * step + warp * kChunk, lane, d);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        keep[v] = add(keep[v], other[v]);
        store8<VEC>(p.h + row * p.d, v * step + warp * kChunk, lane, d, keep[v]);
      }
    }
    if (NORM) {
#pragma unroll
      for (int v = 0; v < NV; ++v) square(keep[v]);
    }
  } else if (NORM) {
    for (int v = 0; v < nstep; ++v) {
      const int c0 = v * step + warp * kChunk;
      uint4 t = load8<VEC>(x, c0, lane, d);
      if (p.res != nullptr) {
        t = add(t, load8<VEC>(res, c0, lane, d));
        store8<VEC>(p.h + row * p.d, c0, lane, d, t);
      }
      square(t);
    }
  }
  float rstd = 1.0f;
  if (NORM) {
    rstd = rsqrtf(fmaf(group_sum<false>(sum[0] + sum[1], s_red + 32 * threadIdx.y, warps), p.inv_d, p.eps));
    if (live && threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int v = 0; v < nstep; ++v) {
    const int c0 = v * step + warp * kChunk;
    if (c0 >= width) break;
    uint4 t;
    if constexpr (NV > 0) {
      t = keep[v];
    } else {
      // the values that this thread wrote or read above
      t = load8<VEC>(NORM && p.res != nullptr ? p.h + row * p.d : x, c0, lane, d);
    }
    float f[8];
    if (NORM) {
      const uint4 g = load8<VEC>(p.gamma, c0, lane, width);
      const uint32_t tw[4] = {t.x, t.y, t.z, t.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = fma_lo(tw[i], gw[i], -0.0f) * rstd;        // -0: a product of zero keeps its sign
        f[2 * i + 1] = fma_hi(tw[i], gw[i], -0.0f) * rstd;
      }
    } else {
      unpack8(t, f);
    }
    if (OUT == kOutBf16)
      store8<VEC>(p.y + row * p.d, c0, lane, d, pack8(f));
    else
      store_fp8<VEC, OUT == kOutE5M2 ? kE5M2 : kE4M3>(p.codes + row * p.ld, p.scales + row * p.nblk, c0, lane, d, f);
  }
}

// Gradients. A CTA of up to 512 threads holds groups of T threads; each takes
// rows of its own, at its own pace: where one waits for its row sum the others
// compute (with one barrier for the CTA's two groups 4096 rows of 4096 took
// 33.0 us, now 27). A thread's columns are the same in every row, so its share of
// dgamma stays in registers until the CTA's groups are added up through shared
// memory, in a fixed order, into one partial row a CTA; k_dgamma adds the
// CTAs' rows.
//
// BULK (rows of whole 16-byte pieces that fit): the rows come through a ring
// of p.stages stages a group in shared memory, filled by bulk copies, and are
// read from there twice, for the row sum and for the output. The barrier of a
// row's sum shows that the group is done with the row before; one thread then
// refills its stage. Otherwise (odd widths, and NV == 0: wide rows, whose
// partial row is kept in global memory) plain loads.
template <int NV, bool VEC, bool BULK>
__global__ void __launch_bounds__(512, 1) k_rmsnorm_bwd(NormBwd p) {
  extern __shared__ __align__(16) uint8_t s_dyn[];   // BULK: the stages; then d floats for the groups' dgamma
  __shared__ float s_red[2][16 * 16];
  __shared__ __align__(8) uint64_t s_bar[16 * ring_words(kBwdMaxStages)];
  static_assert(!BULK || (VEC && NV > 0), "bulk copies are for whole rows in registers");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  constexpr int KEEP = NV > 0 ? NV : 1;
  const int width = static_cast<int>(p.d);
  const int step = warps * kChunk;
  const int nstep = NV > 0 ? NV : (width + step - 1) / step;
  const int groups = static_cast<int>(blockDim.y);
  const bool one = threadIdx.x == 0;     // of a group
  const uint32_t row_bytes = static_cast<uint32_t>(width) * 2;
  const int parts = p.dres != nullptr ? 3 : 2;
  const uint32_t stage_bytes = 3 * row_bytes;
  const uint32_t base = smem_u32(s_dyn) + threadIdx.y * p.stages * stage_bytes;
  BulkRing ring(smem_u32(s_bar) + threadIdx.y * ring_words(kBwdMaxStages) * 8);
  uint64_t acc[KEEP][4];
#pragma unroll
  for (int v = 0; v < KEEP; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[v][i] = 0;
  if (BULK && one) ring.init(p.stages);
  if (BULK) __syncthreads();
  grid_dependency_wait();
  grid_dependency_trigger();
  float* prow = p.part == nullptr ? nullptr : p.part + blockIdx.x * p.d;

  const int64_t stride = static_cast<int64_t>(gridDim.x) * groups;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.y;
  auto fill = [&](int64_t row, int stage) {          // one thread of the group
    if (row >= p.rows || ring.given_up()) return;
    const uint32_t bar = ring.bar(stage), dst = base + stage * stage_bytes;
    ring.expect(stage, parts * row_bytes);
    bulk_load(dst, p.dy + row * p.d, row_bytes, bar);
    bulk_load(dst + row_bytes, p.h + row * p.d, row_bytes, bar);
    if (parts == 3) bulk_load(dst + 2 * row_bytes, p.dres + row * p.d, row_bytes, bar);
  };
  if (BULK && one)
    for (int i = 0; i < p.stages; ++i) fill(row0 + i * stride, i);
  uint4 kg[KEEP];
  if constexpr (NV > 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) kg[v] = load8<VEC>(p.gamma, v * step + warp * kChunk, lane, width);
  }

  int stage = 0, turn = 0;
  float next_rstd = row0 < p.rows ? p.rstd[row0] : 0.0f;
  for (int64_t row = row0; row < p.rows; row += stride) {
    const int d = width;
    const __nv_bfloat16* dy = p.dy + row * p.d;
    const __nv_bfloat16* h = p.h + row * p.d;
    const float rstd = next_rstd;       // fetched a row ahead
    if (row + stride < p.rows) next_rstd = p.rstd[row + stride];
    uint4 kdy[KEEP], kh[KEEP], kres[KEEP];
    float dot = 0.0f;
    const uint32_t src = base + stage * stage_bytes;
    if constexpr (BULK) {
      ring.wait(stage);                 // given up on: this and the later rows are void, the barriers are met
    } else if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c0 = v * step + warp * kChunk;
        kdy[v] = load8<VEC>(dy, c0, lane, d);
        kh[v] = load8<VEC>(h, c0, lane, d);
        if (parts == 3) kres[v] = load8<VEC>(p.dres + row * p.d, c0, lane, d);
      }
    }
    // part 0 dy, 1 h, 2 dres: this lane's 8 values of a chunk
    auto fetch = [&](int part, int v, int c0) -> uint4 {
      if constexpr (BULK) {
        const int c = c0 + 8 * lane;
        return c < d ? lds_u4(src + part * row_bytes + 2 * c) : make_uint4(0, 0, 0, 0);
      } else if constexpr (NV > 0) {
        return part == 0 ? kdy[v] : part == 1 ? kh[v] : kres[v];
      } else {
        return load8<VEC>(part == 0 ? dy : part == 1 ? h : p.dres + row * p.d, c0, lane, d);
      }
    };
    auto gain = [&](int v, int c0) -> uint4 {
      return NV > 0 ? kg[NV > 0 ? v : 0] : load8<VEC>(p.gamma, c0, lane, width);
    };
#pragma unroll
    for (int v = 0; v < nstep; ++v) {
      const int c0 = v * step + warp * kChunk;
      const uint4 a = fetch(0, v, c0), b = fetch(1, v, c0), g = gain(v, c0);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dot = fmaf(fma_lo(aw[i], gw[i], 0.0f), bf_lo(bw[i]), dot);
        dot = fmaf(fma_hi(aw[i], gw[i], 0.0f), bf_hi(bw[i]), dot);
      }
    }
    // two buffers in turn: a warp that is a row ahead does not overwrite sums still being read
    dot = group_sum<true>(dot, s_red[turn] + warps * threadIdx.y, warps);
    turn ^= 1;
    if (BULK && one && row > row0) fill(row + (p.stages - 1) * stride, stage == 0 ? p.stages - 1 : stage - 1);
    // dx = (dy g) rstd - h c + dres, dgamma += (dy rstd) h
    const float c = dot * p.inv_d * rstd * rstd * rstd;
    const uint64_t rstd2 = f2(rstd, rstd), c2 = f2(-c, -c);
#pragma unroll
    for (int v = 0; v < nstep; ++v) {
      const int c0 = v * step + warp * kChunk;
      const uint4 a = fetch(0, v, c0), b = fetch(1, v, c0), g = gain(v, c0);
      const uint4 r = parts == 3 ? fetch(2, v, c0) : make_uint4(0, 0, 0, 0);
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w}, gw[4] = {g.x, g.y, g.z, g.w},
                     rw[4] = {r.x, r.y, r.z, r.w};
      uint32_t o[4];
      uint64_t grad[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t b2 = f2(bf_lo(bw[i]), bf_hi(bw[i]));
        const uint64_t ag = f2(fma_lo(aw[i], gw[i], 0.0f), fma_hi(aw[i], gw[i], 0.0f));
        const uint64_t x2 = f2_fma(ag, rstd2, f2_fma(b2, c2, f2(bf_lo(rw[i]), bf_hi(rw[i]))));
        uint32_t lo, hi;
        f2_split(x2, lo, hi);
        o[i] = pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
        grad[i] = f2_mul(f2_mul(f2(bf_lo(aw[i]), bf_hi(aw[i])), rstd2), b2);
      }
      store8<VEC>(p.dx + row * p.d, c0, lane, d, make_uint4(o[0], o[1], o[2], o[3]));
      if (NV > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[NV > 0 ? v : 0][i] = f2_add(acc[NV > 0 ? v : 0][i], grad[i]);
      } else if (prow != nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = c0 + (VEC ? 8 * lane + j : lane + 32 * j);
          uint32_t lo, hi;
          f2_split(grad[j >> 1], lo, hi);
          if (col < d) prow[col] = __uint_as_float(j & 1 ? hi : lo) + (row == row0 ? 0.0f : prow[col]);
        }
      }
    }
    if (BULK && ++stage == p.stages) stage = 0;
  }
  if (BULK && one) ring.drain();
  if constexpr (NV > 0) {
    if (prow == nullptr) return;
    float* s_part = reinterpret_cast<float*>(s_dyn);
    __syncthreads();                    // the stages are read: their memory takes the groups' sums
    for (int y = 0; y < groups; ++y) {
      if (static_cast<int>(threadIdx.y) == y) {
        const bool last = y + 1 == groups;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int c0 = v * step + warp * kChunk;
          float own[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            f2_split(acc[v][i], lo, hi);
            own[2 * i] = __uint_as_float(lo);
            own[2 * i + 1] = __uint_as_float(hi);
          }
          if (VEC) {
            const int col = c0 + 8 * lane;
            if (col >= width) continue;
#pragma unroll
            for (int h = 0; h < 8; h += 4) {
              float4 t = make_float4(own[h], own[h + 1], own[h + 2], own[h + 3]);
              if (y > 0) {
                const float4 o = *reinterpret_cast<const float4*>(s_part + col + h);
                t = make_float4(o.x + t.x, o.y + t.y, o.z + t.z, o.w + t.w);
              }
              *reinterpret_cast<float4*>((last ? prow : s_part) + col + h) = t;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int col = c0 + lane + 32 * j;
              if (col < width) (last ? prow : s_part)[col] = (y > 0 ? s_part[col] : 0.0f) + own[j];
            }
          }
        }
      }
      __syncthreads();
    }
  }
}

// dgamma[c] = sum over the partial rows, in a fixed order: 32 columns a CTA, 32
// threads a column, so that every load is in flight at once.
__global__ void __launch_bounds__(1024) k_dgamma(const float* __restrict__ part, int nrows, int64_t d, float* dgamma) {
  __shared__ float s[32][33];
  grid_dependency_wait();
  grid_dependency_trigger();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int r = threadIdx.y; r < nrows; r += 32) v += part[r * d + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  v = warp_sum(s[threadIdx.x][threadIdx.y]);      // warp y: column y
  const int64_t out = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < d) dgamma[out] = v;
}

// ------------------------------------------------------------------ host
using host::aligned;
using host::cdiv;
using host::rup;

template <bool VEC, int OUT, bool NORM>
int launch_rows(const NormFwd& p, int sms, cudaStream_t st) {
  // up to four chunks a warp (32 values a thread), so that the sums and
  // scales' fixed cost is shared by many values; short rows share a CTA of 256
  // threads
  // (4096 rows of 8192: 40.2 us, with two chunks 48.2) -- and two where few
  // rows leave SMs idle, since latency counts then (1 row of 4096: 2.4 us, with four 3.0)
  const int few = p.rows < 8 * static_cast<int64_t>(sms) ? 2 : 4;
  const int nv = p.d <= kChunk ? 1 : p.d <= few * 16 * kChunk ? (p.d <= 8 * kChunk ? 2 : few)
                                   : p.d <= 4 * 16 * kChunk ? 4 : 0;
  const int t = nv == 0 ? 1024 : static_cast<int>(cdiv(p.d, int64_t(kChunk) * nv)) * 32;
  const int r = t >= 256 ? 1 : 256 / t;
  const dim3 grid(static_cast<unsigned>(cdiv(p.rows, r))), block(t, r);
  switch (nv) {
    case 1: return host::launch_pdl(k_rows_fwd<1, VEC, OUT, NORM>, grid, block, 0, st, 1, p);
    case 2: return host::launch_pdl(k_rows_fwd<2, VEC, OUT, NORM>, grid, block, 0, st, 1, p);
    case 4: return host::launch_pdl(k_rows_fwd<4, VEC, OUT, NORM>, grid, block, 0, st, 1, p);
    default: return host::launch_pdl(k_rows_fwd<0, VEC, OUT, NORM>, grid, block, 0, st, 1, p);
  }
}

template <int OUT, bool NORM>
int launch_rows_vec(const NormFwd& p, int sms, cudaStream_t st) {
  return p.d % 8 == 0 ? launch_rows<true, OUT, NORM>(p, sms, st) : launch_rows<false, OUT, NORM>(p, sms, st);
}

// The backward's CTA: T threads a row, as many groups as 512 threads hold, and
// as many bulk stages a group (three rows each) as fit, at least two.
struct BwdPlan {
  int nv, t, r;
  int grid;
  int stages;
};

BwdPlan plan_bwd(int64_t rows, int64_t d, int sms) {
  BwdPlan b;
  // four chunks a warp only through bulk stages: without them the rows do not fit the registers
  const int most = d % 8 == 0 ? 4 : 2;
  b.nv = d <= kChunk ? 1 : d <= 2 * kChunk ? 2 : d <= most * 16 * kChunk ? most : 0;
  b.t = b.nv == 0 ? 512 : static_cast<int>(cdiv(d, int64_t(kChunk) * b.nv)) * 32;
  b.r = b.nv == 0 ? 1 : std::max(1, 512 / b.t);
  b.grid = static_cast<int>(std::min<int64_t>(sms, cdiv(rows, b.r)));
  b.stages = b.nv > 0 && d % 8 == 0
                 ? static_cast<int>(std::min<int64_t>(kBwdMaxStages, kBwdMaxSmem / (static_cast<int64_t>(b.r) * 6 * d)))
                 : 0;
  if (b.stages < 2) b.stages = 0;
  return b;
}

template <int NV, bool VEC, bool BULK>
int launch_bwd_nv(const BwdPlan& b, const NormBwd& p, cudaStream_t st) {
  const size_t sums = NV > 0 && b.r > 1 ? static_cast<size_t>(p.d) * sizeof(float) : 0;
  const size_t smem = std::max(static_cast<size_t>(b.stages) * b.r * 6 * p.d, sums);
  return host::launch_pdl(k_rmsnorm_bwd<NV, VEC, BULK>, dim3(b.grid), dim3(b.t, b.r), smem, st, 1, p);
}

int launch_bwd(const BwdPlan& b, const NormBwd& p, cudaStream_t st) {
  if (b.stages > 0) {
    switch (b.nv) {
      case 1: return launch_bwd_nv<1, true, true>(b, p, st);
      case 2: return launch_bwd_nv<2, true, true>(b, p, st);
      default: return launch_bwd_nv<4, true, true>(b, p, st);
    }
  }
  if (p.d % 8 == 0) return launch_bwd_nv<0, true, false>(b, p, st);
  switch (b.nv) {
    case 1: return launch_bwd_nv<1, false, false>(b, p, st);
    case 2: return launch_bwd_nv<2, false, false>(b, p, st);
    default: return launch_bwd_nv<0, false, false>(b, p, st);
  }
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxCols = kFp8MaxCols;

}  // namespace

cudaError_t set_norm_attributes() {
  const int n = static_cast<int>(kBwdMaxSmem);
  cudaError_t e = cudaFuncSetAttribute(k_rmsnorm_bwd<1, true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_rmsnorm_bwd<2, true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_rmsnorm_bwd<4, true, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
  return e;
}

qlora_status_t check_fp8_rows(const qlora_fp8_rows_t* r) {
  if (r == nullptr || r->reserved != 0) return QLORA_ERR_INVALID_ARG;
  if (r->format != QLORA_FP8_E4M3 && r->format != QLORA_FP8_E5M2) return QLORA_ERR_INVALID_ARG;
  if (r->rows < 0 || r->rows > kMaxRows || r->cols < 1 || r->cols > kMaxCols) return QLORA_ERR_SHAPE;
  if (r->ld < r->cols || r->ld % 16 != 0) return QLORA_ERR_SHAPE;
  if (r->rows == 0) return QLORA_OK;
  if (r->codes == nullptr || r->scales == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(r->codes, 16) || !aligned(r->scales, 4)) return QLORA_ERR_ALIGNMENT;
  return QLORA_OK;
}

// Rows to 8 bits (arguments checked by the caller).
int launch_quantize_rows(const void* x_bf16, const qlora_fp8_rows_t& out, int sms, cudaStream_t st) {
  NormFwd p{};
  p.x = static_cast<const __nv_bfloat16*>(x_bf16);
  p.codes = out.codes;
  p.scales = out.scales;
  p.rows = out.rows;
  p.d = out.cols;
  p.ld = out.ld;
  p.nblk = cdiv(out.cols, kFp8Block);
  return out.format == QLORA_FP8_E5M2 ? launch_rows_vec<kOutE5M2, false>(p, sms, st)
                                      : launch_rows_vec<kOutE4M3, false>(p, sms, st);
}

}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status_t qlora_quantize_fp8_rows(const void* x_bf16, const qlora_fp8_rows_t* out, void* stream) {
  qlora_status_t s = check_fp8_rows(out);
  if (s != QLORA_OK || out->rows == 0) return s;
  if (x_bf16 == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16)) return QLORA_ERR_ALIGNMENT;
  int sms = 0;
  if ((s = static_cast<qlora_status_t>(check_current_device(OpFamily::kNorm, &sms))) != QLORA_OK) return s;
  return static_cast<qlora_status_t>(launch_quantize_rows(x_bf16, *out, sms, static_cast<cudaStream_t>(stream)));
}

qlora_status_t qlora_rmsnorm_fwd(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                                 int64_t d, float eps, void* h_out_bf16, void* y_bf16, const qlora_fp8_rows_t* y8,
                                 float* rstd_out, void* stream) {
  if (rows < 0 || rows > kMaxRows || d < 1 || d > kMaxCols) return QLORA_ERR_SHAPE;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return QLORA_ERR_INVALID_ARG;
  if (y8 != nullptr) {
    const qlora_status_t s = check_fp8_rows(y8);
    if (s != QLORA_OK) return s;
    if (y8->rows != rows || y8->cols != d) return QLORA_ERR_SHAPE;
  }
  if (rows == 0) return QLORA_OK;
  if (x_bf16 == nullptr || gamma_bf16 == nullptr || (y_bf16 == nullptr) == (y8 == nullptr) ||
      (residual_bf16 == nullptr) != (h_out_bf16 == nullptr))
    return QLORA_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(gamma_bf16, 16) || !aligned(h_out_bf16, 16) ||
      !aligned(y_bf16, 16) || !aligned(rstd_out, 4))
    return QLORA_ERR_ALIGNMENT;
  int sms = 0;
  const qlora_status_t s = static_cast<qlora_status_t>(check_current_device(OpFamily::kNorm, &sms));
  if (s != QLORA_OK) return s;
  NormFwd p{};
  p.x = static_cast<const __nv_bfloat16*>(x_bf16);
  p.res = static_cast<const __nv_bfloat16*>(residual_bf16);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma_bf16);
  p.h = static_cast<__nv_bfloat16*>(h_out_bf16);
  p.y = static_cast<__nv_bfloat16*>(y_bf16);
  p.rstd = rstd_out;
  p.rows = rows;
  p.d = d;
  p.eps = eps;
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(d));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (y8 == nullptr) return static_cast<qlora_status_t>(launch_rows_vec<kOutBf16, true>(p, sms, st));
  p.codes = y8->codes;
  p.scales = y8->scales;
  p.ld = y8->ld;
  p.nblk = cdiv(d, kFp8Block);
  return static_cast<qlora_status_t>(y8->format == QLORA_FP8_E5M2 ? launch_rows_vec<kOutE5M2, true>(p, sms, st)
                                                                  : launch_rows_vec<kOutE4M3, true>(p, sms, st));
}

size_t qlora_rmsnorm_workspace_bytes(int64_t rows, int64_t d) {
  if (rows < 1 || rows > kMaxRows || d < 1 || d > kMaxCols) return 0;
  int sms = 0;
  if (check_current_device(OpFamily::kNorm, &sms) != QLORA_OK) sms = 148;
  return static_cast<size_t>(plan_bwd(rows, d, sms).grid) * static_cast<size_t>(d) * sizeof(float);
}

qlora_status_t qlora_rmsnorm_bwd(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16, const float* rstd,
                                 const void* dres_bf16, int64_t rows, int64_t d, void* dx_bf16, float* dgamma,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || rows > kMaxRows || d < 1 || d > kMaxCols) return QLORA_ERR_SHAPE;
  if (!aligned(dgamma, 16)) return QLORA_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  qlora_status_t s;
  int sms = 0;
  const dim3 rblock(32, 32), rgrid(static_cast<unsigned>(cdiv(d, 32)));
  if (rows == 0) {
    if (dgamma == nullptr) return QLORA_OK;
    if ((s = static_cast<qlora_status_t>(check_current_device(OpFamily::kNorm, &sms))) != QLORA_OK) return s;
    return static_cast<qlora_status_t>(
        host::launch_pdl(k_dgamma, rgrid, rblock, 0, st, 1, static_cast<const float*>(nullptr), 0, d, dgamma));
  }
  if (dy_bf16 == nullptr || h_bf16 == nullptr || gamma_bf16 == nullptr || rstd == nullptr || dx_bf16 == nullptr)
    return QLORA_ERR_INVALID_ARG;
  if (!aligned(dy_bf16, 16) || !aligned(h_bf16, 16) || !aligned(gamma_bf16, 16) || !aligned(rstd, 4) ||
      !aligned(dres_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(ws, 16))
    return QLORA_ERR_ALIGNMENT;
  if ((s = static_cast<qlora_status_t>(check_current_device(OpFamily::kNorm, &sms))) != QLORA_OK) return s;
  const BwdPlan b = plan_bwd(rows, d, sms);
  if (dgamma != nullptr && (ws == nullptr || ws_bytes < static_cast<size_t>(b.grid) * d * sizeof(float)))
    return QLORA_ERR_WORKSPACE;
  NormBwd p{};
  p.dy = static_cast<const __nv_bfloat16*>(dy_bf16);
  p.h = static_cast<const __nv_bfloat16*>(h_bf16);
  p.gamma = static_cast<const __nv_bfloat16*>(gamma_bf16);
  p.rstd = rstd;
  p.dres = static_cast<const __nv_bfloat16*>(dres_bf16);
  p.dx = static_cast<__nv_bfloat16*>(dx_bf16);
  p.part = dgamma == nullptr ? nullptr : static_cast<float*>(ws);
  p.rows = rows;
  p.d = d;
  p.inv_d = static_cast<float>(1.0 / static_cast<double>(d));
  p.stages = b.stages;
  s = static_cast<qlora_status_t>(launch_bwd(b, p, st));
  if (s != QLORA_OK || dgamma == nullptr) return s;
  return static_cast<qlora_status_t>(host::launch_pdl(k_dgamma, rgrid, rblock, 0, st, 1,
                                                      static_cast<const float*>(ws), b.grid, d, dgamma));
}

}  // extern "C"
