// RMS norm with the residual's addition, and its gradients (sm_100a).
//
//   h = bf16(x + res);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd gamma
//   dx = rstd (dy g - h rstd^2 mean(dy g h)) + dres;  dgamma = sum_rows dy h rstd
//
// Both are streams over the rows, bound by HBM bandwidth (7 bytes a value
// forward with a residual and 8-bit output, 8 backward with a residual), so a
// row is read once and stays in registers between its statistics and its
// output. A group of T threads owns a row; warps own chunks of 256 columns.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "fp8_dev.cuh"
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
  float eps;
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
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A lane's 8 values of a chunk. VEC: columns c0 + 8 lane + j, one 16-byte
// access (d % 8 == 0); else columns c0 + lane + 32 j, so that 2-byte accesses
// of a warp fall into one line. Packed as bf16 pairs (2i, 2i + 1).
template <bool VEC>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int64_t c0, int lane, int64_t d) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (VEC) {
    const int64_t c = c0 + 8 * lane;
    if (c < d) v = *reinterpret_cast<const uint4*>(row + c);
  } else {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = c0 + lane + 32 * j;
      w[j] = c < d ? p[c] : 0u;
    }
    v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  return v;
}

template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int64_t c0, int lane, int64_t d, uint4 v) {
  if (VEC) {
    const int64_t c = c0 + 8 * lane;
    if (c < d) *reinterpret_cast<uint4*>(row + c) = v;
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(row);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t c = c0 + lane + 32 * j;
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
__device__ __forceinline__ void store_fp8(uint8_t* row, float* scales, int64_t c0, int lane, int64_t d, int64_t nblk,
                                          const float (&f)[8]) {
  constexpr float F = fp8_top<FMT>();
  const int64_t b0 = c0 / kFp8Block;
  if (VEC) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fp8_mag(f[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
    a = fmaxf(a, kFp8Least);
    const float inv = F / a;
    const int64_t c = c0 + 8 * lane;
    if (c < d) {
      uint2 q;
      q.x = fp8_pack4<FMT>(fp8_scaled(f[0], inv), fp8_scaled(f[1], inv), fp8_scaled(f[2], inv), fp8_scaled(f[3], inv));
      q.y = fp8_pack4<FMT>(fp8_scaled(f[4], inv), fp8_scaled(f[5], inv), fp8_scaled(f[6], inv), fp8_scaled(f[7], inv));
      *reinterpret_cast<uint2*>(row + c) = q;
      if ((lane & 15) == 0) scales[b0 + (lane >> 4)] = a / F;
    }
  } else {
    float a[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j >> 2] = fmaxf(a[j >> 2], fp8_mag(f[j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a[0] = fmaxf(a[0], __shfl_xor_sync(0xFFFFFFFFu, a[0], o));
      a[1] = fmaxf(a[1], __shfl_xor_sync(0xFFFFFFFFu, a[1], o));
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      a[b] = fmaxf(a[b], kFp8Least);
      const float inv = F / a[b];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t c = c0 + lane + 32 * (4 * b + j);
        const float s = fp8_scaled(f[4 * b + j], inv);
        if (c < d) row[c] = static_cast<uint8_t>(fp8_pack2<FMT>(s, s));
      }
      if (lane == 0 && b0 + b < nblk) scales[b0 + b] = a[b] / F;
    }
  }
}

// Sum over the T threads of a row group (threadIdx.y); `red` has 32 floats a group.
__device__ __forceinline__ float group_sum(float v, float* red, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[w] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.0f);
}

enum NormOut : int { kOutBf16 = 0, kOutE4M3 = 1, kOutE5M2 = 2 };

// NV chunks a warp, kept in registers; NV == 0: any width, h is read again
// for the output (rows of over 32768 values).
// NORM false: the rows are only quantized (y = x).
template <int NV, bool VEC, int OUT, bool NORM>
__global__ void __launch_bounds__(1024) k_rows_fwd(NormFwd p) {
  __shared__ float s_red[32 * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = row < p.rows;
  const int64_t d = live ? p.d : 0;     // an idle group reads and writes nothing
  const __nv_bfloat16* x = p.x + row * p.d;
  const __nv_bfloat16* res = p.res + row * p.d;
  constexpr int KEEP = NV > 0 ? NV : 1;
  const int64_t step = static_cast<int64_t>(warps) * kChunk;
  const int64_t nstep = NV > 0 ? NV : (p.d + step - 1) / step;
  uint4 keep[KEEP];
  grid_dependency_wait();
  grid_dependency_trigger();

  auto add = [&](uint4 a, uint4 b) {
    float fa[8], fb[8];
    unpack8(a, fa);
    unpack8(b, fb);
#pragma unroll
    for (int j = 0; j < 8; ++j) fa[j] += fb[j];
    return pack8(fa);
  };
  float sum = 0.0f;
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
      for (int v = 0; v < NV; ++v) {
        float f[8];
        unpack8(keep[v], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
      }
    }
  } else if (NORM) {
    for (int64_t v = 0; v < nstep; ++v) {
      const int64_t c0 = v * step + warp * kChunk;
      uint4 t = load8<VEC>(x, c0, lane, d);
      if (p.res != nullptr) {
        t = add(t, load8<VEC>(res, c0, lane, d));
        store8<VEC>(p.h + row * p.d, c0, lane, d, t);
      }
      float f[8];
      unpack8(t, f);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
    }
  }
  float rstd = 1.0f;
  if (NORM) {
    sum = group_sum(sum, s_red + 32 * threadIdx.y, warps);
    rstd = 1.0f / sqrtf(sum / static_cast<float>(p.d) + p.eps);
    if (live && threadIdx.x == 0 && p.rstd != nullptr) p.rstd[row] = rstd;
  }
#pragma unroll
  for (int64_t v = 0; v < nstep; ++v) {
    const int64_t c0 = v * step + warp * kChunk;
    if (c0 >= p.d) break;
    uint4 t;
    if constexpr (NV > 0) {
      t = keep[v];
    } else {
      // the values that this thread wrote or read above
      t = load8<VEC>(NORM && p.res != nullptr ? p.h + row * p.d : x, c0, lane, d);
    }
    float f[8];
    unpack8(t, f);
    if (NORM) {
      float g[8];
      unpack8(load8<VEC>(p.gamma, c0, lane, p.d), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * g[j];
    }
    if (OUT == kOutBf16)
      store8<VEC>(p.y + row * p.d, c0, lane, d, pack8(f));
    else
      store_fp8<VEC, OUT == kOutE5M2 ? kE5M2 : kE4M3>(p.codes + row * p.ld, p.scales + row * p.nblk, c0, lane, d,
                                                      live ? p.nblk : 0, f);
  }
}

// Gradients. A CTA of up to 512 threads holds groups of T threads; group y
// takes rows y, y + groups, ... A thread's columns are the same in every row,
// so its share of dgamma stays in registers until the CTA's groups are added
// up through shared memory, in a fixed order, into one partial row a CTA;
// k_dgamma adds the CTAs' rows. NV == 0: any width, the partial row is kept in
// global memory (one group a CTA, each thread its own columns).
template <int NV, bool VEC>
__global__ void __launch_bounds__(512, 1) k_rmsnorm_bwd(NormBwd p) {
  extern __shared__ float s_part[];      // NV > 0 and more than one group: d floats
  __shared__ float s_red[2][16 * 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  constexpr int KEEP = NV > 0 ? NV : 1;
  const int64_t step = static_cast<int64_t>(warps) * kChunk;
  const int64_t nstep = NV > 0 ? NV : (p.d + step - 1) / step;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * blockDim.y;
  const float inv_d = 1.0f / static_cast<float>(p.d);
  float acc[KEEP][8];
#pragma unroll
  for (int v = 0; v < KEEP; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.0f;
  grid_dependency_wait();
  grid_dependency_trigger();
  float* prow = p.part == nullptr ? nullptr : p.part + blockIdx.x * p.d;

  // every group of the CTA runs the same number of rounds: the barrier of the
  // row sum is the whole CTA's
  const int64_t rounds = (p.rows + groups - 1) / groups;
  for (int64_t i = 0; i < rounds; ++i) {
    const int64_t row = (i * gridDim.x + blockIdx.x) * blockDim.y + threadIdx.y;
    const bool live = row < p.rows;
    const int64_t d = live ? p.d : 0;
    const __nv_bfloat16* dy = p.dy + row * p.d;
    const __nv_bfloat16* h = p.h + row * p.d;
    const float rstd = live ? p.rstd[row] : 0.0f;
    uint4 kdy[KEEP], kh[KEEP], kres[KEEP];
    float dot = 0.0f;
    if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int64_t c0 = v * step + warp * kChunk;
        kdy[v] = load8<VEC>(dy, c0, lane, d);
        kh[v] = load8<VEC>(h, c0, lane, d);
        if (p.dres != nullptr) kres[v] = load8<VEC>(p.dres + row * p.d, c0, lane, d);
      }
    }
#pragma unroll
    for (int64_t v = 0; v < nstep; ++v) {
      const int64_t c0 = v * step + warp * kChunk;
      float a[8], b[8], g[8];
      unpack8(NV > 0 ? kdy[NV > 0 ? v : 0] : load8<VEC>(dy, c0, lane, d), a);
      unpack8(NV > 0 ? kh[NV > 0 ? v : 0] : load8<VEC>(h, c0, lane, d), b);
      unpack8(load8<VEC>(p.gamma, c0, lane, p.d), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = fmaf(a[j] * g[j], b[j], dot);
    }
    // two buffers in turn: a warp that is a round ahead does not overwrite sums still being read
    dot = group_sum(dot, s_red[i & 1] + 16 * threadIdx.y, warps);
    const float c = dot * inv_d * rstd * rstd;
#pragma unroll
    for (int64_t v = 0; v < nstep; ++v) {
      const int64_t c0 = v * step + warp * kChunk;
      float a[8], b[8], g[8], o[8];
      unpack8(NV > 0 ? kdy[NV > 0 ? v : 0] : load8<VEC>(dy, c0, lane, d), a);
      unpack8(NV > 0 ? kh[NV > 0 ? v : 0] : load8<VEC>(h, c0, lane, d), b);
      unpack8(load8<VEC>(p.gamma, c0, lane, p.d), g);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = (a[j] * g[j] - b[j] * c) * rstd;
      if (p.dres != nullptr) {
        float r[8];
        unpack8(NV > 0 ? kres[NV > 0 ? v : 0] : load8<VEC>(p.dres + row * p.d, c0, lane, d), r);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += r[j];
      }
      store8<VEC>(p.dx + row * p.d, c0, lane, d, pack8(o));
      if (NV > 0) {
        if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[NV > 0 ? v : 0][j] = fmaf(a[j], b[j] * rstd, acc[NV > 0 ? v : 0][j]);
        }
      } else if (prow != nullptr && live) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int64_t col = c0 + (VEC ? 8 * lane + j : lane + 32 * j);
          if (col < d) prow[col] = fmaf(a[j], b[j] * rstd, i == 0 ? 0.0f : prow[col]);
        }
      }
    }
  }
  if constexpr (NV > 0) {
    if (prow == nullptr) return;
    for (int y = 0; y < static_cast<int>(blockDim.y); ++y) {
      if (static_cast<int>(threadIdx.y) == y) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int64_t col = v * step + warp * kChunk + (VEC ? 8 * lane + j : lane + 32 * j);
            if (col < p.d) {
              const float t = y == 0 ? acc[v][j] : s_part[col] + acc[v][j];
              if (y + 1 < static_cast<int>(blockDim.y))
                s_part[col] = t;
              else
                prow[col] = t;
            }
          }
      }
      __syncthreads();
    }
  }
}

// dgamma[c] = sum over the partial rows, in a fixed order: 32 columns a CTA,
// eight threads a column.
__global__ void __launch_bounds__(256) k_dgamma(const float* __restrict__ part, int nrows, int64_t d, float* dgamma) {
  __shared__ float s[8][33];
  grid_dependency_wait();
  grid_dependency_trigger();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < d) {
#pragma unroll 8
    for (int r = threadIdx.y; r < nrows; r += 8) v += part[r * d + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < d) {
    for (int y = 1; y < 8; ++y) v += s[y][threadIdx.x];
    dgamma[c] = v;
  }
}

// ------------------------------------------------------------------ host
using host::aligned;
using host::cdiv;
using host::rup;

template <bool VEC, int OUT, bool NORM>
int launch_rows(const NormFwd& p, cudaStream_t st) {
  // two chunks a warp (16 values a thread) once the row is wide enough; short
  // rows share a CTA of 256 threads
  const int nv = p.d <= kChunk ? 1 : p.d <= 2 * 32 * kChunk ? 2 : p.d <= 4 * 32 * kChunk ? 4 : 0;
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
int launch_rows_vec(const NormFwd& p, cudaStream_t st) {
  return p.d % 8 == 0 ? launch_rows<true, OUT, NORM>(p, st) : launch_rows<false, OUT, NORM>(p, st);
}

// The backward's CTA: T threads a row, as many groups as 512 threads hold.
struct BwdPlan {
  int nv, t, r;
  int grid;
};

BwdPlan plan_bwd(int64_t rows, int64_t d, int sms) {
  BwdPlan b;
  b.nv = d <= kChunk ? 1 : d <= 2 * 16 * kChunk ? 2 : d <= 4 * 16 * kChunk ? 4 : 0;
  b.t = b.nv == 0 ? 512 : static_cast<int>(cdiv(d, int64_t(kChunk) * b.nv)) * 32;
  b.r = b.nv == 0 ? 1 : std::max(1, 512 / b.t);
  b.grid = static_cast<int>(std::min<int64_t>(sms, cdiv(rows, b.r)));
  return b;
}

template <int NV, bool VEC>
int launch_bwd_nv(const BwdPlan& b, const NormBwd& p, cudaStream_t st) {
  const size_t smem = NV > 0 && b.r > 1 ? static_cast<size_t>(p.d) * sizeof(float) : 0;
  return host::launch_pdl(k_rmsnorm_bwd<NV, VEC>, dim3(b.grid), dim3(b.t, b.r), smem, st, 1, p);
}

template <bool VEC>
int launch_bwd(const BwdPlan& b, const NormBwd& p, cudaStream_t st) {
  switch (b.nv) {
    case 1: return launch_bwd_nv<1, VEC>(b, p, st);
    case 2: return launch_bwd_nv<2, VEC>(b, p, st);
    case 4: return launch_bwd_nv<4, VEC>(b, p, st);
    default: return launch_bwd_nv<0, VEC>(b, p, st);
  }
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

}  // namespace

qlora_status_t check_fp8_rows(const qlora_fp8_rows_t* r) {
  if (r == nullptr || r->reserved != 0) return QLORA_ERR_INVALID_ARG;
  if (r->format != QLORA_FP8_E4M3 && r->format != QLORA_FP8_E5M2) return QLORA_ERR_INVALID_ARG;
  if (r->rows < 0 || r->rows > kMaxRows || r->cols < 1 || r->cols > kMaxRows) return QLORA_ERR_SHAPE;
  if (r->ld < r->cols || r->ld % 16 != 0) return QLORA_ERR_SHAPE;
  if (r->rows == 0) return QLORA_OK;
  if (r->codes == nullptr || r->scales == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(r->codes, 16) || !aligned(r->scales, 4)) return QLORA_ERR_ALIGNMENT;
  return QLORA_OK;
}

// Rows to 8 bits (arguments checked by the caller).
int launch_quantize_rows(const void* x_bf16, const qlora_fp8_rows_t& out, cudaStream_t st) {
  NormFwd p{};
  p.x = static_cast<const __nv_bfloat16*>(x_bf16);
  p.codes = out.codes;
  p.scales = out.scales;
  p.rows = out.rows;
  p.d = out.cols;
  p.ld = out.ld;
  p.nblk = cdiv(out.cols, kFp8Block);
  return out.format == QLORA_FP8_E5M2 ? launch_rows_vec<kOutE5M2, false>(p, st)
                                      : launch_rows_vec<kOutE4M3, false>(p, st);
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
  if ((s = static_cast<qlora_status_t>(check_current_device(&sms))) != QLORA_OK) return s;
  return static_cast<qlora_status_t>(launch_quantize_rows(x_bf16, *out, static_cast<cudaStream_t>(stream)));
}

qlora_status_t qlora_rmsnorm_fwd(const void* x_bf16, const void* residual_bf16, const void* gamma_bf16, int64_t rows,
                                 int64_t d, float eps, void* h_out_bf16, void* y_bf16, const qlora_fp8_rows_t* y8,
                                 float* rstd_out, void* stream) {
  if (rows < 0 || rows > kMaxRows || d < 1 || d > kMaxRows) return QLORA_ERR_SHAPE;
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
  const qlora_status_t s = static_cast<qlora_status_t>(check_current_device(&sms));
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (y8 == nullptr) return static_cast<qlora_status_t>(launch_rows_vec<kOutBf16, true>(p, st));
  p.codes = y8->codes;
  p.scales = y8->scales;
  p.ld = y8->ld;
  p.nblk = cdiv(d, kFp8Block);
  return static_cast<qlora_status_t>(y8->format == QLORA_FP8_E5M2 ? launch_rows_vec<kOutE5M2, true>(p, st)
                                                                  : launch_rows_vec<kOutE4M3, true>(p, st));
}

size_t qlora_rmsnorm_workspace_bytes(int64_t rows, int64_t d) {
  if (rows < 1 || rows > kMaxRows || d < 1 || d > kMaxRows) return 0;
  int sms = 0;
  if (check_current_device(&sms) != QLORA_OK) sms = 148;
  return static_cast<size_t>(plan_bwd(rows, d, sms).grid) * static_cast<size_t>(d) * sizeof(float);
}

qlora_status_t qlora_rmsnorm_bwd(const void* dy_bf16, const void* h_bf16, const void* gamma_bf16, const float* rstd,
                                 const void* dres_bf16, int64_t rows, int64_t d, void* dx_bf16, float* dgamma,
                                 void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || rows > kMaxRows || d < 1 || d > kMaxRows) return QLORA_ERR_SHAPE;
  if (!aligned(dgamma, 16)) return QLORA_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  qlora_status_t s;
  int sms = 0;
  const dim3 rblock(32, 8), rgrid(static_cast<unsigned>(cdiv(d, 32)));
  if (rows == 0) {
    if (dgamma == nullptr) return QLORA_OK;
    if ((s = static_cast<qlora_status_t>(check_current_device(&sms))) != QLORA_OK) return s;
    return static_cast<qlora_status_t>(
        host::launch_pdl(k_dgamma, rgrid, rblock, 0, st, 1, static_cast<const float*>(nullptr), 0, d, dgamma));
  }
  if (dy_bf16 == nullptr || h_bf16 == nullptr || gamma_bf16 == nullptr || rstd == nullptr || dx_bf16 == nullptr)
    return QLORA_ERR_INVALID_ARG;
  if (!aligned(dy_bf16, 16) || !aligned(h_bf16, 16) || !aligned(gamma_bf16, 16) || !aligned(rstd, 4) ||
      !aligned(dres_bf16, 16) || !aligned(dx_bf16, 16) || !aligned(ws, 16))
    return QLORA_ERR_ALIGNMENT;
  if ((s = static_cast<qlora_status_t>(check_current_device(&sms))) != QLORA_OK) return s;
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
  s = static_cast<qlora_status_t>(d % 8 == 0 ? launch_bwd<true>(b, p, st) : launch_bwd<false>(b, p, st));
  if (s != QLORA_OK || dgamma == nullptr) return s;
  return static_cast<qlora_status_t>(host::launch_pdl(k_dgamma, rgrid, rblock, 0, st, 1,
                                                      static_cast<const float*>(ws), b.grid, d, dgamma));
}

}  // extern "C"
