// The CTA-pair kernel of the 8-bit product.
#pragma once

#include "fp8_gemm.cuh"

namespace qlora {

constexpr int kFp8PairStages = 5;            // 32 KB each
constexpr int kFp8PairBoxes = 8 * 4 * 2048;  // four 32 x 32 bf16 output boxes an epilogue warp
constexpr int kFp8PairSmem = kFp8PairStages * 32768 + kFp8PairBoxes + 1024 + 256;

// tm_x: rows' codes [m x red], boxes {128, 128}; tm_w: weight codes [N x K],
// boxes {128, 128}, both 128-byte swizzled; tm_out: y [m x cols] bf16, boxes
// {32, 32}, 64-byte swizzled (p.tma_out). Launched in clusters of two.
template <bool W_MN>
__global__ void k_fp8_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_out, Fp8Gemm p);

}  // namespace qlora
