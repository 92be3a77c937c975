// 8-bit linear: weights in e4m3 with one scale per 128 x 128 block, rows in
// e4m3 or e5m2 with one scale per 128 columns (see fp8_dev.cuh).
//
//   y[m][n]  = sum_b sx[m][b] sw[n/128][b] sum_{k in b} x[m][k] w[n][k]
//   dX[m][k] = sum_b sd[m][b] sw[b][k/128] sum_{n in b} d[m][n] w[n][k]
#include <algorithm>
#include <cmath>
#include <cstring>

#include <cuda_bf16.h>

#include "../../include/qlora.h"
#include "fp8_dev.cuh"
#include "fp8_launch.h"
#include "host.h"
#include "ptx.cuh"

namespace qlora {

qlora_status_t check_fp8_rows(const qlora_fp8_rows_t* r);
int launch_quantize_rows(const void* x_bf16, const qlora_fp8_rows_t& out, cudaStream_t st);

namespace {

// ------------------------------------------------------------------ weight quantizer
// One CTA per 128 x 128 block: 8 values a thread and step, 16 steps, kept in
// registers between the maximum and the codes. Bound by HBM (3 bytes a value).
__global__ void __launch_bounds__(256) k_quantize_fp8(const __nv_bfloat16* __restrict__ w, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales, int64_t n, int64_t k) {
  __shared__ float s_max[8];
  const int64_t nbk = (k + kFp8Block - 1) / kFp8Block;
  const int64_t bn = blockIdx.x / nbk, bk = blockIdx.x % nbk;
  const int64_t col = bk * kFp8Block + 8 * (threadIdx.x & 15);
  const int64_t row0 = bn * kFp8Block + (threadIdx.x >> 4);
  uint4 v[8];
  float a = 0.0f;
  grid_dependency_wait();
  grid_dependency_trigger();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i;
    v[i] = make_uint4(0, 0, 0, 0);
    if (row < n && col < k) v[i] = __ldcs(reinterpret_cast<const uint4*>(w + row * k + col));   // k % 16 == 0
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a = fmaxf(a, fp8_mag(__uint_as_float(u[j] << 16)));
      a = fmaxf(a, fp8_mag(__uint_as_float(u[j] & 0xFFFF0000u)));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, s_max[i]);
  constexpr float F = 448.0f;
  a = fmaxf(a, kFp8Least);
  const float inv = F / a;
  if (threadIdx.x == 0) scales[blockIdx.x] = a / F;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 16 * i;
    if (row >= n || col >= k) continue;
    const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = fp8_pack2<kE4M3>(fp8_scaled(__uint_as_float(u[j] << 16), inv),
                              fp8_scaled(__uint_as_float(u[j] & 0xFFFF0000u), inv));
    *reinterpret_cast<uint2*>(codes + row * k + col) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
  }
}

// bf16(code * scale), eight values a thread; rows over blockIdx.y and on.
__global__ void __launch_bounds__(256) k_dequantize_fp8(const uint8_t* __restrict__ codes,
                                                        const float* __restrict__ scales, __nv_bfloat16* __restrict__ w,
                                                        int64_t n, int64_t k) {
  grid_dependency_wait();
  grid_dependency_trigger();
  const int64_t nbk = (k + kFp8Block - 1) / kFp8Block;
  const int64_t total = n * k / 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i * 8 / k, col = i * 8 % k;
    const float s = scales[(row / kFp8Block) * nbk + col / kFp8Block];
    const uint2 q = __ldcs(reinterpret_cast<const uint2*>(codes) + i);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = fp8_unpack2<kE4M3>((j < 2 ? q.x : q.y) >> (16 * (j & 1)));
      o[j] = pack_bf16x2(f.x * s, f.y * s);
    }
    reinterpret_cast<uint4*>(w)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ------------------------------------------------------------------ product
struct Product {
  const uint8_t* x;        // [m x red] codes, ldx bytes from row to row
  const float* sx;         // [m x xblk]
  const uint8_t* w;        // weight codes [N x K]
  const float* sw;         // [ceil(N/128) x nbk]
  __nv_bfloat16* y;        // [m x cols]
  int64_t m, cols, red;    // red: K forward, N backward
  int64_t ldx, xblk, k, nbk;
};

// 64 x 64 outputs a CTA, 16 a thread, the reduction in steps of 32.
template <bool BWD, int FMT>
__global__ void __launch_bounds__(256) k_fp8_product(Product p) {
  __shared__ float sx[32][65], sw[32][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  float acc[4][4] = {}, part[4][4] = {};
  grid_dependency_wait();
  grid_dependency_trigger();
  for (int64_t r0 = 0; r0 < p.red; r0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int a = i >> 5, r = i & 31;
      sx[r][a] = (m0 + a < p.m && r0 + r < p.red) ? fp8_unpack2<FMT>(p.x[(m0 + a) * p.ldx + r0 + r]).x : 0.0f;
      if (!BWD)
        sw[r][a] = (c0 + a < p.cols && r0 + r < p.red) ? fp8_unpack2<kE4M3>(p.w[(c0 + a) * p.k + r0 + r]).x : 0.0f;
    }
    if (BWD)
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        const int a = i & 63, r = i >> 6;
        sw[r][a] = (c0 + a < p.cols && r0 + r < p.red) ? fp8_unpack2<kE4M3>(p.w[(r0 + r) * p.k + c0 + a]).x : 0.0f;
      }
    __syncthreads();
#pragma unroll 8
    for (int r = 0; r < 32; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sx[r][ty + 16 * i], sw[r][tx + 16 * j], part[i][j]);
    __syncthreads();
    if ((r0 + 32) % kFp8Block == 0 || r0 + 32 >= p.red) {
      const int64_t b = r0 / kFp8Block;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + ty + 16 * i, c = c0 + tx + 16 * j;
          if (m < p.m && c < p.cols) {
            const int64_t cb = c / kFp8Block;
            const float s = p.sx[m * p.xblk + b] * p.sw[BWD ? b * p.nbk + cb : cb * p.nbk + b];
            acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
          }
          part[i][j] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, c = c0 + tx + 16 * j;
      if (m < p.m && c < p.cols) p.y[m * p.cols + c] = __float2bfloat16_rn(acc[i][j]);
    }
}

// ------------------------------------------------------------------ host
using host::al256;
using host::aligned;
using host::cdiv;
using host::rup;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

qlora_status_t check_weight(const qlora_fp8_t* q) {
  if (q == nullptr || q->codes == nullptr || q->scales == nullptr) return QLORA_ERR_INVALID_ARG;
  if (q->n_out < 1 || q->k_in < 1 || q->k_in % 16 != 0 || q->n_out > kMaxDim || q->k_in > kMaxDim)
    return QLORA_ERR_SHAPE;
  if (!aligned(q->codes, 16) || !aligned(q->scales, 4)) return QLORA_ERR_ALIGNMENT;
  return QLORA_OK;
}

template <bool BWD>
int launch_pair_product(const Product& p, int format, int pairs, cudaStream_t st) {
  Fp8Gemm g{};
  g.status = device_status_word();
  g.sx = p.sx;
  g.sw = p.sw;
  g.y = p.y;
  g.xblk = p.xblk;
  g.sw_out = BWD ? 1 : p.nbk;
  g.sw_red = BWD ? p.nbk : 1;
  g.m = static_cast<int32_t>(p.m);
  g.cols = static_cast<int32_t>(p.cols);
  g.kblocks = static_cast<int32_t>(p.xblk);
  g.tiles_m = static_cast<int32_t>(cdiv(p.m, 256));
  g.tiles_n = static_cast<int32_t>(cdiv(p.cols, 256));
  g.a_format = format;
  g.tma_out = p.cols % 8 == 0;
  CUtensorMap x, w, o;
  std::memset(&o, 0, sizeof(o));
  const int64_t n = BWD ? p.red : p.cols;
  if (!encode_map2d(&x, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.x, p.red, p.m, p.ldx, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.w, p.k, n, p.k, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
      (g.tma_out && !encode_map2d(&o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.y, p.cols, p.m, p.cols * 2, 32, 32,
                                  CU_TENSOR_MAP_SWIZZLE_64B)))
    return QLORA_ERR_CUDA;
  return launch_fp8_pair(BWD, x, w, o, g, pairs, st);
}

// Workspace of a product over rows of `red` values: the rows' codes and scales.
struct ProductPlan {
  size_t codes, scales, total;
};

ProductPlan plan_product(int64_t m, int64_t red) {
  ProductPlan p;
  p.codes = 0;
  p.scales = al256(static_cast<size_t>(m) * rup(red, 16));
  p.total = p.scales + al256(static_cast<size_t>(m) * cdiv(red, kFp8Block) * sizeof(float));
  return p;
}

template <bool BWD>
qlora_status_t product(const qlora_fp8_t* q, const void* x_bf16, const qlora_fp8_rows_t* x8, int32_t format, int64_t m,
                       void* out_bf16, void* ws, size_t ws_bytes, cudaStream_t st) {
  qlora_status_t s = check_weight(q);
  if (s != QLORA_OK) return s;
  if (format != QLORA_FP8_E4M3 && format != QLORA_FP8_E5M2) return QLORA_ERR_INVALID_ARG;
  if (m < 0 || m > kMaxDim) return QLORA_ERR_SHAPE;
  const int64_t red = BWD ? q->n_out : q->k_in, cols = BWD ? q->k_in : q->n_out;
  if (x8 != nullptr) {
    if ((s = check_fp8_rows(x8)) != QLORA_OK) return s;
    if (x8->rows != m || x8->cols != red) return QLORA_ERR_SHAPE;
  }
  if (m == 0) return QLORA_OK;
  if ((x_bf16 == nullptr) == (x8 == nullptr) || out_bf16 == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(out_bf16, 16) || !aligned(ws, 16)) return QLORA_ERR_ALIGNMENT;
  int sms = 0, pairs = 0;
  if ((s = static_cast<qlora_status_t>(check_current_device(&sms, &pairs))) != QLORA_OK) return s;
  qlora_fp8_rows_t rows;
  if (x8 != nullptr) {
    rows = *x8;
  } else {
    const ProductPlan plan = plan_product(m, red);
    if (ws == nullptr || ws_bytes < plan.total) return QLORA_ERR_WORKSPACE;
    uint8_t* base = static_cast<uint8_t*>(ws);
    rows = qlora_fp8_rows_t{m, red, rup(red, 16), base + plan.codes, reinterpret_cast<float*>(base + plan.scales),
                            format, 0};
    if ((s = static_cast<qlora_status_t>(launch_quantize_rows(x_bf16, rows, st))) != QLORA_OK) return s;
  }
  Product p{rows.codes, rows.scales, q->codes, q->scales, static_cast<__nv_bfloat16*>(out_bf16), m, cols, red,
            rows.ld, cdiv(red, kFp8Block), q->k_in, cdiv(q->k_in, kFp8Block)};
  if (m > 128) return static_cast<qlora_status_t>(launch_pair_product<BWD>(p, rows.format, pairs, st));
  const dim3 grid(static_cast<unsigned>(cdiv(cols, 64)), static_cast<unsigned>(cdiv(m, 64)));
  return static_cast<qlora_status_t>(
      rows.format == QLORA_FP8_E5M2 ? host::launch_pdl(k_fp8_product<BWD, kE5M2>, grid, dim3(256), 0, st, 1, p)
                                    : host::launch_pdl(k_fp8_product<BWD, kE4M3>, grid, dim3(256), 0, st, 1, p));
}

}  // namespace

cudaError_t set_fp8_attributes() { return set_fp8_pair_attributes(); }

}  // namespace qlora

using namespace qlora;

extern "C" {

qlora_status_t qlora_quantize_fp8(const void* w_bf16, const qlora_fp8_t* q, void* stream) {
  qlora_status_t s = check_weight(q);
  if (s != QLORA_OK) return s;
  if (w_bf16 == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(w_bf16, 16)) return QLORA_ERR_ALIGNMENT;
  const int64_t blocks = cdiv(q->n_out, kFp8Block) * cdiv(q->k_in, kFp8Block);
  if (blocks > kMaxDim) return QLORA_ERR_SHAPE;
  int sms = 0;
  if ((s = static_cast<qlora_status_t>(check_current_device(&sms))) != QLORA_OK) return s;
  return static_cast<qlora_status_t>(host::launch_pdl(
      k_quantize_fp8, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<cudaStream_t>(stream), 1,
      static_cast<const __nv_bfloat16*>(w_bf16), q->codes, q->scales, q->n_out, q->k_in));
}

qlora_status_t qlora_dequantize_fp8(const qlora_fp8_t* q, void* w_bf16_out, void* stream) {
  qlora_status_t s = check_weight(q);
  if (s != QLORA_OK) return s;
  if (w_bf16_out == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(w_bf16_out, 16)) return QLORA_ERR_ALIGNMENT;
  int sms = 0;
  if ((s = static_cast<qlora_status_t>(check_current_device(&sms))) != QLORA_OK) return s;
  const int64_t blocks = std::min<int64_t>(cdiv(q->n_out * (q->k_in / 8), 256), int64_t(sms) * 8);
  return static_cast<qlora_status_t>(host::launch_pdl(
      k_dequantize_fp8, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<cudaStream_t>(stream), 1,
      static_cast<const uint8_t*>(q->codes), static_cast<const float*>(q->scales),
      static_cast<__nv_bfloat16*>(w_bf16_out), q->n_out, q->k_in));
}

size_t qlora_fp8_workspace_bytes(int64_t m, int64_t n_out, int64_t k_in) {
  if (m < 1 || m > kMaxDim || n_out < 1 || n_out > kMaxDim || k_in < 1 || k_in > kMaxDim || k_in % 16 != 0) return 0;
  return std::max(plan_product(m, k_in).total, plan_product(m, n_out).total);
}

qlora_status_t qlora_fp8_linear_fwd(const qlora_fp8_t* q, const void* x_bf16, const qlora_fp8_rows_t* x8, int64_t m,
                                    void* y_bf16, void* ws, size_t ws_bytes, void* stream) {
  return product<false>(q, x_bf16, x8, QLORA_FP8_E4M3, m, y_bf16, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

qlora_status_t qlora_fp8_linear_bwd(const qlora_fp8_t* q, const void* dy_bf16, const qlora_fp8_rows_t* dy8,
                                    int32_t format, int64_t m, void* dx_bf16, void* ws, size_t ws_bytes,
                                    void* stream) {
  return product<true>(q, dy_bf16, dy8, format, m, dx_bf16, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
