// 8-bit product on CTA pairs (cta_group::2), sm_100a: the kernel of long inputs.
//
//   D[256 rows x 256 outputs] = sum_b (sx[row][b] sw[output block][b]) X_b[256 x 128] W_b[256 x 128]^T
//
// Both scales change from one block of 128 of the reduction to the next, so
// the tensor core's sum ends with the block: each block's product goes to one
// of two tensor-memory buffers, and the epilogue warps add it, times its
// scales, to the fp32 sums they keep in registers while the tensor core fills
// the other buffer. With rows on the tensor-memory lanes a thread owns one row
// and 128 outputs of one weight block, so the two scales are one factor a
// thread and block. (Scales that are powers of two could go into the tensor
// core itself; these are any fp32 numbers.)
//
// What bounds it: a block takes the tensor core 256 x 128 x 128 multiply-adds
// a SM, 512 cycles at its dense 8-bit rate; reading 128 x 256 sums back takes
// 256 cycles of tensor-memory bandwidth, and as many of fp32 FMAs (half that
// packed in pairs), spread over eight warps. Operands: 32 KB a SM and block,
// each CTA loading its own 128 rows and its own 128 of the 256 outputs.
//
// The weight is read as it lies, [N x K] row-major: K-major for the forward,
// MN-major for dX (W_MN), whose reduction runs along N. In both a stage holds
// 128 rows of 128 bytes in the 128-byte swizzle.
//
// Warps of a CTA (320 threads): 0 TMA; 1 tensor-memory allocation and, in the
// even CTA, the MMA issue; 2-9 epilogue (lane quarter = warp % 4, output half
// = (warp - 2) / 4). Every wait is bounded.
#include "fp8_pair.h"

namespace qlora {

using namespace tcd;

template <bool W_MN>
__global__ void __launch_bounds__(320, 1)
    k_fp8_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_out, Fp8Gemm p) {
  constexpr int STAGES = kFp8PairStages;
  constexpr uint32_t HALF = 16384;                // 128 rows x 128 bytes
  constexpr uint32_t STAGE_BYTES = 2 * HALF;      // this CTA's rows, then its outputs
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t boxes = base + STAGES * STAGE_BYTES;
  const uint32_t bar0 = boxes + kFp8PairBoxes;
  uint8_t* const ctl = smem_raw + (bar0 - raw);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };                  // even CTA: loads of both
  auto bar_empty = [&](int s) { return bar0 + 8u * (STAGES + s); };      // local, from the MMA
  auto bar_accf = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };   // local, from the MMA
  auto bar_acce = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };   // even CTA: 16 epilogue warps
  const uint32_t bar_fin = bar0 + 8u * (2 * STAGES + 4);
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(ctl + 8 * (2 * STAGES + 5));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * (2 * STAGES + 5) + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const bool leader = (rank == 0);
  const int pair = blockIdx.x >> 1;
  const int npairs = gridDim.x >> 1;
  const int ntiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_accf(b), 1);
      mbar_init(bar_acce(b), 16);
    }
    mbar_init(bar_fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();   // barriers initialised and tensor memory allocated in both CTAs
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dependency_wait();
  grid_dependency_trigger();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(&tm_w);
      int it = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < ntiles; tile += npairs) {
        const int row = (tile % p.tiles_m) * 256 + 128 * rank;
        const int out = (tile / p.tiles_m) * 256 + 128 * rank;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % STAGES;
          if (!mbar_wait(bar_empty(s), ((it / STAGES) & 1) ^ 1, abort_flag, QLORA_DEV_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t x_s = base + s * STAGE_BYTES;
          const uint32_t full_even = mapa_shared(bar_full(s), 0);
          if (leader) mbar_arrive_expect_tx(bar_full(s), 2 * STAGE_BYTES);
          tma_load_2d_pair(x_s, &tm_x, full_even, kb * 128, row);
          if (W_MN)
            tma_load_2d_pair(x_s + HALF, &tm_w, full_even, out, kb * 128);
          else
            tma_load_2d_pair(x_s + HALF, &tm_w, full_even, kb * 128, out);
        }
      }
      // the loads this thread started have landed once the MMA released their stage
      for (int j = max(0, it - STAGES); j < it; ++j) drain_wait(bar_empty(j % STAGES), (j / STAGES) & 1);
    }
  } else if (warp == 1) {
    if (leader && lane == 0) {
      const uint32_t idesc = idesc_fp8(256, 256, p.a_format, W_MN);
      int it = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < ntiles; tile += npairs) {
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % STAGES, b = it & 1;
          if (!mbar_wait_cluster(bar_acce(b), ((it >> 1) & 1) ^ 1, abort_flag, QLORA_DEV_TIMEOUT_MMA) ||
              !mbar_wait(bar_full(s), (it / STAGES) & 1, abort_flag, QLORA_DEV_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t x_s = base + s * STAGE_BYTES, w_s = x_s + HALF;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {   // 32 of the reduction each
            const uint64_t dx = smem_desc_sw128(x_s + kk * 32, 16, 1024);
            const uint64_t dw = W_MN ? smem_desc_sw128(w_s + kk * 4096, HALF, 1024)
                                     : smem_desc_sw128(w_s + kk * 32, 16, 1024);
            tc_mma_fp8_pair(tmem_base + b * 256, dx, dw, idesc, kk > 0 ? 1u : 0u);
          }
          tc_commit_pair(bar_empty(s));
          tc_commit_pair(mapa_shared(bar_empty(s), 1));
          tc_commit_pair(bar_accf(b));
          tc_commit_pair(mapa_shared(bar_accf(b), 1));
        }
      }
      tc_commit_pair(bar_fin);
      drain_wait(bar_fin, 0);
    }
  } else {
    const int quarter = warp & 3;               // tensor-memory lanes [32 q, 32 q + 32) belong to warp % 4
    const int half = (warp - 2) >> 2;
    const uint32_t acce_even0 = mapa_shared(bar_acce(0), 0);
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 128 * half;
    const uint32_t box = boxes + (warp - 2) * 8192;
    int it = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < ntiles; tile += npairs) {
      const int row0 = (tile % p.tiles_m) * 256 + 128 * rank + 32 * quarter;
      const int col0 = (tile / p.tiles_m) * 256 + 128 * half;
      const int row = row0 + lane;
      // a row or block past the end has no scale: its products are zero and not stored
      const float* sx = p.sx + static_cast<int64_t>(row) * p.xblk;
      const float* sw = p.sw + static_cast<int64_t>(col0 >> 7) * p.sw_out;
      const bool live_x = row < p.m, live_w = col0 < p.cols;
      float nx = live_x ? __ldg(sx) : 0.0f, nw = live_w ? __ldg(sw) : 0.0f;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const int b = it & 1;
        const float s = nx * nw;
        const uint64_t s2 = f2(s, s);
        if (kb + 1 < p.kblocks) {
          nx = live_x ? __ldg(sx + kb + 1) : 0.0f;
          nw = live_w ? __ldg(sw + (kb + 1) * p.sw_red) : 0.0f;
        }
        ok = mbar_wait(bar_accf(b), (it >> 1) & 1, abort_flag, QLORA_DEV_TIMEOUT_EPI);
        if (!warp_all(ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t = tbase + b * 256;
        uint32_t ra[16], rb[16];
        tmem_ld_32x32b_x16(t, ra);
        tc_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          tmem_ld_32x32b_x16(t + 16 * (c + 1), rb);
          promote16(acc + 8 * c, ra, s2);
          tc_wait_ld();
          if (c + 2 < 8) {
            tmem_ld_32x32b_x16(t + 16 * (c + 2), ra);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(acce_even0 + 8u * b);
          }
          promote16(acc + 8 * (c + 1), rb, s2);
          if (c + 2 < 8) tc_wait_ld();
        }
      }
      if (!ok) break;
      if (p.tma_out) {
        if (lane == 0) bulk_wait_read_all();   // the previous tile's stores have read the boxes
        __syncwarp();
        const uint32_t sw4 = (lane >> 1) & 3;
#pragma unroll
        for (int c = 0; c < 4; ++c) {          // 32 x 32 boxes in the 64-byte swizzle
          const uint32_t dst = box + c * 2048 + lane * 64;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t lo, hi;
              f2_split(acc[16 * c + 4 * v + e], lo, hi);
              pk[e] = pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
            }
            sts128(dst + ((v ^ sw4) << 4), pk[0], pk[1], pk[2], pk[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < p.m) {
          for (int c = 0; c < 4; ++c)
            if (col0 + 32 * c < p.cols) tma_store_2d(&tm_out, box + c * 2048, col0 + 32 * c, row0);
          bulk_commit();
        }
      } else if (row < p.m) {
        __nv_bfloat16* y = p.y + static_cast<int64_t>(row) * p.cols + col0;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          uint32_t lo, hi;
          f2_split(acc[i], lo, hi);
          if (col0 + 2 * i < p.cols) y[2 * i] = __float2bfloat16_rn(__uint_as_float(lo));
          if (col0 + 2 * i + 1 < p.cols) y[2 * i + 1] = __float2bfloat16_rn(__uint_as_float(hi));
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // stores complete before the CTA's shared memory goes away
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // no CTA leaves while its pair still reads its shared or tensor memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template __global__ void k_fp8_pair<false>(const __grid_constant__ CUtensorMap, const __grid_constant__ CUtensorMap,
                                           const __grid_constant__ CUtensorMap, Fp8Gemm);
template __global__ void k_fp8_pair<true>(const __grid_constant__ CUtensorMap, const __grid_constant__ CUtensorMap,
                                          const __grid_constant__ CUtensorMap, Fp8Gemm);

}  // namespace qlora
