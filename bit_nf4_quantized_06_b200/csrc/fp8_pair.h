// The CTA-pair kernel of the 8-bit product.
#pragma once

#include "fp8_gemm.cuh"

namespace qlora {

constexpr int kFp8PairStages = 4;            // 32 KB each
constexpr int kFp8PairThreads = 640;         // TMA, MMA and two scale warps; 16 epilogue warps
constexpr int kFp8PairIssueRegs = 32, kFp8PairEpiRegs = 112;
// 640 threads are launched with at most 96 registers each
static_assert(128 * kFp8PairIssueRegs + 512 * kFp8PairEpiRegs <= 640 * 96, "registers of the launch");
constexpr int kFp8PairBoxes = 16 * 2 * 2048; // two 32 x 32 bf16 output boxes an epilogue warp
// scales: two chunks of eight reduction blocks, each block 128 rows' and two
// weight blocks' (132 words: a warp's transposed stores spread over the banks)
constexpr int kScaleChunk = 8, kScaleStride = 132;
constexpr int kFp8PairRing = 2 * kScaleChunk * kScaleStride * 4;
constexpr int kFp8PairSmem = kFp8PairStages * 32768 + kFp8PairBoxes + kFp8PairRing + 1024 + 256;

// tm_x: rows' codes [m x red], boxes {128, 128}; tm_w: weight codes [N x K],
// boxes {128, 128}, both 128-byte swizzled; tm_out: y [m x cols] bf16, boxes
// {32, 32}, 64-byte swizzled (p.tma_out). Launched in clusters of two.
template <bool W_MN>
__global__ void k_fp8_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                           const __grid_constant__ CUtensorMap tm_out, Fp8Gemm p);

}  // namespace qlora
