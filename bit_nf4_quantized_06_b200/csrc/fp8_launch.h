// Parameters and launches of the 8-bit product's tensor-core kernels.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace qlora {

struct Fp8Gemm {
  unsigned int* status;     // the library's device status word
  const float* sx;          // [m x xblk] scales of the rows
  const float* sw;          // scales of the weight, at output block * sw_out + reduction block * sw_red
  __nv_bfloat16* y;         // [m x cols]
  int64_t xblk, sw_out, sw_red;
  int32_t m, cols;
  int32_t kblocks;          // reduction blocks of 128
  int32_t tiles_m, tiles_n;
  int32_t a_format;         // format of the rows' codes (Fp8Format)
  int32_t tma_out;          // output rows are 16-byte aligned (cols % 8 == 0)
  // split kernel
  int32_t splits;           // CTAs of a cluster that share a tile's reduction
  int32_t box_m;            // rows of tm_x's boxes
  int32_t early_w;          // the kernel in front has waited for everything before it
  const __nv_bfloat16* x16; // up to kFp8QuantRows bf16 rows [m x red] (red % 8 == 0), quantized in the kernel; else null
  int64_t red;
};

// CTA-pair kernel (fp8_pair.cu). tm_x: rows' codes [m x red], boxes
// {128, 128}; tm_w: weight codes [N x K], boxes {128, 128}, both 128-byte
// swizzled; tm_out: y [m x cols] bf16, boxes {32, 32}, 64-byte swizzled
// (p.tma_out). `w_mn`: the reduction runs along N (dX).
int launch_fp8_pair(bool w_mn, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_out,
                    const Fp8Gemm& p, int pairs, cudaStream_t st);
cudaError_t set_fp8_pair_attributes();

// Split kernel (fp8_split.cu): 128 x 128 tiles, the reduction over clusters
// of p.splits (1 to kFp8MaxSplits, at most the number of blocks). tm_x: boxes {128,
// p.box_m} (unused with p.x16); tm_w: boxes {128, 128}.
int launch_fp8_split(bool w_mn, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const Fp8Gemm& p, cudaStream_t st);
cudaError_t set_fp8_split_attributes(int dev);
constexpr int kFp8MaxSplits = 8;
constexpr int64_t kFp8MaxCols = int64_t(1) << 30;   // of a row: columns are 32-bit numbers in the kernels
constexpr int kFp8QuantRows = 4;
// How many clusters of `splits` CTAs fit on device `dev` at once.
int fp8_split_clusters(int dev, int splits);

}  // namespace qlora
