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
int launch_quantize_rows(const void* x_bf16, const qlora_fp8_rows_t& out, int sms, cudaStream_t st);

namespace {

// ------------------------------------------------------------------ weight quantizer
// One CTA per 128 x 128 block: 8 values a thread and step, eight steps, kept in
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

// bf16(code * scale), eight values a thread and step, the weight as one list.
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

struct Product {
  qlora_fp8_rows_t x;      // [m x red]
  const void* x16;         // bf16 rows to quantize within the product, or null
  const qlora_fp8_t* q;
  void* y;                 // [m x cols]
  int64_t m, cols, red;    // red: K forward, N backward
  bool quantized_here;     // the rows' quantizer is the kernel in front
};

// The tile shape and the split, by an estimate of the time in microseconds.
// Measured on B200 with rows already in 8 bits:
//   pair kernel   5 + waves (1.5 + 0.40 blocks): 512 rows x 4096 x 4096 17.8, 1024 rows 18.9, 2048 rows 33.6
//   split kernel  waves (4.7 + 0.004 S rows + (0.2 + 0.0006 rows) ceil(blocks / S)), a wave being
//                 the clusters of S CTAs that are resident at once:
//                 4096 x 4096 weight, 1 row: 10.6 (S = 1), 7.2 (2), 6.0 (4), 13.5 (8, two waves);
//                 128 rows: 12.9, 9.7, 8.4, 21.9; 512 rows, S = 1: 13.5; 1024 rows: 26.9
struct Choice {
  bool pair;
  int splits;
};

Choice choose(int64_t m, int64_t cols, int64_t kblocks, int dev, int pairs) {
  const double blocks = static_cast<double>(kblocks);
  const int64_t pair_waves = cdiv(cdiv(m, 256) * cdiv(cols, 256), pairs);
  Choice best{true, 1};
  double best_cost = 5.0 + static_cast<double>(pair_waves) * (1.5 + 0.40 * blocks);
  const int64_t tiles = cdiv(m, 128) * cdiv(cols, 128);
  const double rows = static_cast<double>(std::min<int64_t>(m, 128));
  for (int s = 1; s <= kFp8MaxSplits && s <= kblocks && tiles * s < (int64_t(1) << 30); ++s) {
    const int resident = fp8_split_clusters(dev, s);
    if (resident < 1) continue;
    const double waves = static_cast<double>(cdiv(tiles, resident));
    const double cost = waves * (4.7 + (s > 1 ? 0.004 * s * rows : 0.0) +
                                 (0.2 + 0.0006 * rows) * static_cast<double>(cdiv(kblocks, s)));
    if (cost < best_cost) {
      best_cost = cost;
      best = Choice{false, s};
    }
  }
  return best;
}

template <bool BWD>
int launch_product(const Product& p, int dev, int pairs, cudaStream_t st) {
  const qlora_fp8_t& q = *p.q;
  const int64_t nbk = cdiv(q.k_in, kFp8Block);
  Fp8Gemm g{};
  g.status = device_status_word();
  g.sx = p.x.scales;
  g.sw = q.scales;
  g.y = static_cast<__nv_bfloat16*>(p.y);
  g.xblk = cdiv(p.red, kFp8Block);
  g.sw_out = BWD ? 1 : nbk;
  g.sw_red = BWD ? nbk : 1;
  g.m = static_cast<int32_t>(p.m);
  g.cols = static_cast<int32_t>(p.cols);
  g.kblocks = static_cast<int32_t>(g.xblk);
  g.a_format = p.x.format;
  g.tma_out = p.cols % 8 == 0;
  if (cdiv(p.m, 256) * cdiv(p.cols, 256) > (int64_t(1) << 30)) return QLORA_ERR_SHAPE;   // tile numbers are 32-bit
  const Choice c = choose(p.m, p.cols, g.xblk, dev, pairs);
  g.x16 = static_cast<const __nv_bfloat16*>(p.x16);
  g.red = p.red;
  const int tile = c.pair ? 256 : 128;
  g.tiles_m = static_cast<int32_t>(cdiv(p.m, tile));
  g.tiles_n = static_cast<int32_t>(cdiv(p.cols, tile));
  g.splits = c.splits;
  g.box_m = c.pair ? 128 : static_cast<int32_t>(std::min<int64_t>(128, rup(p.m, 8)));
  g.early_w = p.quantized_here;
  CUtensorMap x, w, o;
  std::memset(&o, 0, sizeof(o));
  std::memset(&x, 0, sizeof(x));
  if ((g.x16 == nullptr && !encode_map2d(&x, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.x.codes, p.red, p.m, p.x.ld, 128,
                                         g.box_m, CU_TENSOR_MAP_SWIZZLE_128B)) ||
      !encode_map2d(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, q.codes, q.k_in, q.n_out, q.k_in, 128, 128,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return QLORA_ERR_CUDA;
  if (!c.pair) return launch_fp8_split(BWD, x, w, g, st);
  if (g.tma_out && !encode_map2d(&o, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.y, p.cols, p.m, p.cols * 2, 32, 32,
                                 CU_TENSOR_MAP_SWIZZLE_64B))
    return QLORA_ERR_CUDA;
  return launch_fp8_pair(BWD, x, w, o, g, pairs, st);
}

// Whether a product quantizes its bf16 rows itself: few rows of whole 16-byte
// pieces, where the split kernel runs.
bool quantizes(int64_t m, int64_t cols, int64_t red, int dev, int pairs) {
  return m <= kFp8QuantRows && red % 8 == 0 && !choose(m, cols, cdiv(red, kFp8Block), dev, pairs).pair;
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
  if (x8 == nullptr && format != QLORA_FP8_E4M3 && format != QLORA_FP8_E5M2) return QLORA_ERR_INVALID_ARG;
  if (m < 0 || m > kMaxDim) return QLORA_ERR_SHAPE;
  const int64_t red = BWD ? q->n_out : q->k_in, cols = BWD ? q->k_in : q->n_out;
  if (x8 != nullptr) {
    if ((s = check_fp8_rows(x8)) != QLORA_OK) return s;
    if (x8->rows != m || x8->cols != red) return QLORA_ERR_SHAPE;
  } else if (red > kFp8MaxCols) {
    return QLORA_ERR_SHAPE;      // what check_fp8_rows says of rows in 8 bits
  }
  if (m == 0) return QLORA_OK;
  if ((x_bf16 == nullptr) == (x8 == nullptr) || out_bf16 == nullptr) return QLORA_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(out_bf16, 16) || !aligned(ws, 16)) return QLORA_ERR_ALIGNMENT;
  int sms = 0, pairs = 0;
  if ((s = static_cast<qlora_status_t>(check_current_device(OpFamily::kFp8, &sms, &pairs))) != QLORA_OK) return s;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return QLORA_ERR_CUDA;
  qlora_fp8_rows_t rows;
  const bool within = x8 == nullptr && quantizes(m, cols, red, dev, pairs);
  if (x8 != nullptr) {
    rows = *x8;
  } else if (within) {
    rows = qlora_fp8_rows_t{m, red, red, nullptr, nullptr, format, 0};
  } else {
    const ProductPlan plan = plan_product(m, red);
    if (ws == nullptr || ws_bytes < plan.total) return QLORA_ERR_WORKSPACE;
    uint8_t* base = static_cast<uint8_t*>(ws);
    rows = qlora_fp8_rows_t{m, red, rup(red, 16), base + plan.codes, reinterpret_cast<float*>(base + plan.scales),
                            format, 0};
    if ((s = static_cast<qlora_status_t>(launch_quantize_rows(x_bf16, rows, sms, st))) != QLORA_OK) return s;
  }
  const Product p{rows, within ? x_bf16 : nullptr, q, out_bf16, m, cols, red, x8 == nullptr && !within};
  return static_cast<qlora_status_t>(launch_product<BWD>(p, dev, pairs, st));
}

}  // namespace

cudaError_t set_fp8_attributes(int dev) {
  const cudaError_t e = set_fp8_pair_attributes();
  return e == cudaSuccess ? set_fp8_split_attributes(dev) : e;
}

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
  if ((s = static_cast<qlora_status_t>(check_current_device(OpFamily::kFp8, &sms))) != QLORA_OK) return s;
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
  if ((s = static_cast<qlora_status_t>(check_current_device(OpFamily::kFp8, &sms))) != QLORA_OK) return s;
  const int64_t blocks = std::min<int64_t>(cdiv(q->n_out * (q->k_in / 8), 256), int64_t(sms) * 8);
  return static_cast<qlora_status_t>(host::launch_pdl(
      k_dequantize_fp8, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<cudaStream_t>(stream), 1,
      static_cast<const uint8_t*>(q->codes), static_cast<const float*>(q->scales),
      static_cast<__nv_bfloat16*>(w_bf16_out), q->n_out, q->k_in));
}

size_t qlora_fp8_workspace_bytes(int64_t m, int64_t n_out, int64_t k_in) {
  if (m < 1 || m > kMaxDim || n_out < 1 || n_out > kMaxDim || k_in < 1 || k_in > kMaxDim || k_in % 16 != 0) return 0;
  int dev = 0, sms = 0, pairs = 0;
  if (m <= kFp8QuantRows && check_current_device(OpFamily::kFp8, &sms, &pairs) == QLORA_OK && cudaGetDevice(&dev) == cudaSuccess &&
      quantizes(m, n_out, k_in, dev, pairs) && quantizes(m, k_in, n_out, dev, pairs))
    return 0;
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
