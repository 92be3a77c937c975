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
// Measured, 4096 rows x 11008 outputs x 4096: 189 us, 1.95 PFLOP/s, at the
// board's 1000 W limit (SM clock 1.6 of 1.965 GHz; single launches with pauses
// 166 us); dX of the same weight 200 us with the rows' quantizer. A block takes
// some 890 cycles, where the tensor core needs 512. Its sums are ready 740 after
// the issue, and the epilogue warps take 450 to read them back and free the
// buffer: with two buffers that alone would allow a block every 595 cycles, so
// it is not what holds the kernel by itself. With the epilogue's FMAs taken out
// in a copy a block still takes 690: the operands' way (L2 at 50 bytes a clock
// and SM, then load, MMA and release through four stages) holds it there, and
// the epilogue costs the other 200. How many stages would shorten the first part
// was not measured. On the way: scales read by the epilogue
// warps themselves 275 us; sixteen epilogue warps and one line of shared memory a
// scale 222; eight with 216 registers 211; barrier waits taken ahead 192; a
// chunk's scales read at once 190, the MMA's thread spinning 189. Not kept, all slower: tiles of 160 outputs
// with three buffers (206, dX 232) and of 192 with twelve epilogue warps (213):
// more operand bytes an output; halves of 128 outputs with four buffers (220);
// 32 columns a load, the next block's first ones requested ahead (195); one
// barrier arrival a CTA instead of one a warp (229).
//
// Warps of a CTA (384 threads): 0 TMA; 1 tensor-memory allocation and, in the
// even CTA, the MMA issue; 2-3 scales; 4-11 epilogue (lane quarter = warp % 4,
// output half = (warp - 4) / 4). Every wait is bounded.
#include <algorithm>

#include "fp8_gemm.cuh"
#include "host.h"

namespace qlora {
namespace {

using namespace tcd;

constexpr int kFp8PairStages = 4;            // 32 KB each
constexpr int kFp8PairThreads = 384;         // TMA, MMA and two scale warps; 8 epilogue warps
constexpr int kFp8PairIssueRegs = 56, kFp8PairEpiRegs = 216;
// 384 threads are launched with at most 168 registers each
static_assert(128 * kFp8PairIssueRegs + 256 * kFp8PairEpiRegs <= 384 * 168, "registers of the launch");
constexpr int kFp8PairBoxes = 8 * 4 * 2048;  // four 32 x 32 bf16 output boxes an epilogue warp
// scales: two chunks of eight reduction blocks, each 128 rows of eight (48
// bytes apart: eight lanes' 16-byte loads then take all banks) and two weight
// blocks' eight
constexpr int kScaleChunk = 8, kScaleRow = 48;
constexpr int kScaleBytes = 128 * kScaleRow + 2 * 4 * kScaleChunk;
constexpr int kFp8PairRing = 2 * kScaleBytes;
constexpr int kFp8PairSmem = kFp8PairStages * 32768 + kFp8PairBoxes + kFp8PairRing + 1024 + 256;


template <bool W_MN>
__global__ void __launch_bounds__(kFp8PairThreads, 1)
    k_fp8_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ CUtensorMap tm_out, Fp8Gemm p) {
  constexpr int STAGES = kFp8PairStages;
  constexpr uint32_t HALF = 16384;                // 128 rows x 128 bytes
  constexpr uint32_t STAGE_BYTES = 2 * HALF;      // this CTA's rows, then its outputs
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t boxes = base + STAGES * STAGE_BYTES;
  const uint32_t ring = boxes + kFp8PairBoxes;
  const uint32_t bar0 = ring + kFp8PairRing;
  uint8_t* const ctl = smem_raw + (bar0 - raw);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };                  // even CTA: loads of both
  auto bar_empty = [&](int s) { return bar0 + 8u * (STAGES + s); };      // local, from the MMA
  auto bar_accf = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };   // local, from the MMA
  auto bar_acce = [&](int b) { return bar0 + 8u * (2 * STAGES + 2 + b); };   // even CTA: 16 epilogue warps
  auto bar_sf = [&](int c) { return bar0 + 8u * (2 * STAGES + 4 + c); };     // two scale warps
  auto bar_se = [&](int c) { return bar0 + 8u * (2 * STAGES + 6 + c); };     // 8 epilogue warps
  const uint32_t bar_fin = bar0 + 8u * (2 * STAGES + 8);
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(ctl + 8 * (2 * STAGES + 9));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(ctl + 8 * (2 * STAGES + 9) + 4);
  const Fp8Abort ab{abort_flag, p.status};

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
      mbar_init(bar_sf(b), 2);
      mbar_init(bar_se(b), 8);
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

  // registers move from the first warpgroup to the epilogue's two (the three
  // shares' sum stays below the launch's)
  if (warp < 4) setmaxnreg_dec<kFp8PairIssueRegs>();
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
          if (!fp8_wait(bar_empty(s), ((it / STAGES) & 1) ^ 1, ab, QLORA_DEV_TIMEOUT_PRODUCER)) {
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
    if (leader && elect_one()) {
      const uint32_t idesc = idesc_fp8(256, 256, p.a_format, W_MN);
      const uint64_t dx0 = smem_desc_sw128(base, 16, 1024);
      const uint64_t dw0 = W_MN ? smem_desc_sw128(base + HALF, HALF, 1024) : smem_desc_sw128(base + HALF, 16, 1024);
      int s = 0, b = 0;
      uint32_t ph = 0, aph = 1;     // parities of the stage and of the buffer
      bool full = false, free = false;
      const int64_t blocks = static_cast<int64_t>((ntiles - pair + npairs - 1) / npairs) * p.kblocks;
      for (int64_t i = 0; i < blocks; ++i) {
        if (!full && !fp8_wait(bar_full(s), ph, ab, QLORA_DEV_TIMEOUT_MMA)) break;
        if (!free && !fp8_spin(bar_acce(b), aph, ab, QLORA_DEV_TIMEOUT_MMA)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + b * 256, accf = bar_accf(b), empty = bar_empty(s);
        const uint64_t dx = dx0 + s * (STAGE_BYTES >> 4), dw = dw0 + s * (STAGE_BYTES >> 4);
        if (++s == STAGES) {
          s = 0;
          ph ^= 1;
        }
        b ^= 1;
        if (b == 0) aph ^= 1;
        full = fp8_token(bar_full(s), ph);
        free = fp8_token(bar_acce(b), aph);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 32 of the reduction each
          tc_mma_fp8_pair(d, dx + kk * 2, dw + kk * (W_MN ? 256 : 2), idesc, kk > 0 ? 1u : 0u);
        tc_commit_both(accf);
        tc_commit_both(empty);
      }
      tc_commit_pair(bar_fin);
      drain_wait(bar_fin, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    // scales: chunks of eight reduction blocks, a slot holding each row's eight
    // together and then the two weight blocks' eight each; a warp reads four
    // rows of eight at a time from memory, and an epilogue thread its row's
    // eight in two 16-byte loads. A chunk is requested while the one before is at work: its loads wait in
    // registers for the slot (requested only once the slot was free, they held
    // the epilogue up by 320 to 700 cycles a block).
    const int half = warp - 2;                  // rows [64 half, 64 half + 64)
    const int kl = lane & 7, rl = lane >> 3;
    float v[16], w = 0.0f;
    auto request = [&](int tile, int k0) {
      const int row0 = (tile % p.tiles_m) * 256 + 128 * rank + 64 * half + rl;
      const int ob = (tile / p.tiles_m) * 2 + half;          // this warp's weight block
      const int kb = k0 + kl;
      const bool live = tile < ntiles && kb < p.kblocks;
      const float* sx = p.sx + static_cast<int64_t>(row0) * p.xblk + kb;
#pragma unroll
      for (int j = 0; j < 16; ++j)      // a row or block past the end has scale zero
        v[j] = (live && row0 + 4 * j < p.m) ? __ldg(sx + 4 * j * p.xblk) : 0.0f;
      w = (live && rl == 0 && ob * 128 < p.cols) ? __ldg(p.sw + ob * p.sw_out + kb * p.sw_red) : 0.0f;
    };
    int c = 0;
    uint32_t cph = 1;
    int tile = pair, k0 = 0;
    request(tile, k0);
    while (tile < ntiles && !__any_sync(0xFFFFFFFFu, *abort_flag)) {
      const uint32_t slot = ring + c * kScaleBytes + 4 * kl;
      if (!fp8_token(bar_se(c), cph)) fp8_wait(bar_se(c), cph, ab, QLORA_DEV_TIMEOUT_PRODUCER);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) sts32(slot + (64 * half + rl + 4 * j) * kScaleRow, __float_as_uint(v[j]));
      if (rl == 0) sts32(slot + 128 * kScaleRow + 4 * kScaleChunk * half, __float_as_uint(w));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sf(c));
      c ^= 1;
      if (c == 0) cph ^= 1;
      k0 += kScaleChunk;
      if (k0 >= p.kblocks) {
        k0 = 0;
        tile += npairs;
      }
      request(tile, k0);
    }
  } else {
    setmaxnreg_inc<kFp8PairEpiRegs>();
    const int quarter = warp & 3;               // tensor-memory lanes [32 q, 32 q + 32) belong to warp % 4
    const int half = (warp - 4) >> 2;           // 128 of the 256 outputs: one weight block
    const uint32_t acce_even0 = mapa_shared(bar_acce(0), 0);
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 128 * half;
    const uint32_t box = boxes + (warp - 4) * 8192;
    const uint32_t ring_x = ring + (32 * quarter + lane) * kScaleRow;
    const uint32_t ring_w = ring + 128 * kScaleRow + 4 * kScaleChunk * half;
    int b = 0, c = 0;              // accumulator buffer, scale chunk buffer
    uint32_t bph = 0, cph = 0;     // their parities
    bool ready = false;            // token of bar_accf(b)
    for (int tile = pair; tile < ntiles; tile += npairs) {
      if (__any_sync(0xFFFFFFFFu, *abort_flag)) break;
      const int row0 = (tile % p.tiles_m) * 256 + 128 * rank + 32 * quarter;
      const int col0 = (tile / p.tiles_m) * 256 + 128 * half;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
#pragma unroll 1
      for (int k0 = 0; k0 < p.kblocks; k0 += kScaleChunk) {
        // the chunk's factors, all at once: a round trip through shared memory in
        // every block would hold its sums up
        if (!fp8_token(bar_sf(c), cph)) fp8_wait(bar_sf(c), cph, ab, QLORA_DEV_TIMEOUT_EPI);
        __syncwarp();
        float s[kScaleChunk];
#pragma unroll
        for (int h = 0; h < kScaleChunk; h += 4) {
          const float4 x = lds_f4(ring_x + c * kScaleBytes + 4 * h), w = lds_f4(ring_w + c * kScaleBytes + 4 * h);
          s[h] = x.x * w.x;
          s[h + 1] = x.y * w.y;
          s[h + 2] = x.z * w.z;
          s[h + 3] = x.w * w.w;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_se(c));
        c ^= 1;
        if (c == 0) cph ^= 1;
#pragma unroll 1
        for (int kb = min(p.kblocks - k0, kScaleChunk); kb > 0; --kb) {
          const uint64_t s2 = f2(s[0], s[0]);
#pragma unroll
          for (int j = 0; j + 1 < kScaleChunk; ++j) s[j] = s[j + 1];
          if (!ready) fp8_wait(bar_accf(b), bph, ab, QLORA_DEV_TIMEOUT_EPI);
          __syncwarp();
          tc_fence_after();
          const uint32_t t = tbase + b * 256;
          const uint32_t acce = acce_even0 + 8u * b;
          b ^= 1;
          if (b == 0) bph ^= 1;
          uint32_t ra[16], rb[16];
          tmem_ld_32x32b_x16(t, ra);
          tmem_ld_32x32b_x16(t + 16, rb);
          ready = fp8_token(bar_accf(b), bph);
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            tc_wait_ld();
            if (i == 6) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster(acce);
            }
            promote16(acc + 8 * i, ra, s2);
            if (i < 6) tmem_ld_32x32b_x16(t + 16 * (i + 2), ra);
            promote16(acc + 8 * (i + 1), rb, s2);
            if (i < 6) tmem_ld_32x32b_x16(t + 16 * (i + 3), rb);
          }
        }
      }
      if (p.tma_out) {
        if (lane == 0) bulk_wait_read_all();   // the previous tile's stores have read the boxes
        __syncwarp();
        const uint32_t sw4 = (lane >> 1) & 3;
#pragma unroll
        for (int c4 = 0; c4 < 4; ++c4) {       // 32 x 32 boxes in the 64-byte swizzle
          const uint32_t dst = box + c4 * 2048 + lane * 64;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t pk[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t lo, hi;
              f2_split(acc[16 * c4 + 4 * v + e], lo, hi);
              pk[e] = pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
            }
            sts128(dst + ((v ^ sw4) << 4), pk[0], pk[1], pk[2], pk[3]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && row0 < p.m) {
          for (int c4 = 0; c4 < 4; ++c4)
            if (col0 + 32 * c4 < p.cols) tma_store_2d(&tm_out, box + c4 * 2048, col0 + 32 * c4, row0);
          bulk_commit();
        }
      } else {
        // rows that are not 16-byte aligned: through the same memory (16-byte
        // pieces, the row's low bits exchanged into the piece's), then a row a
        // warp, so that a store is one contiguous piece (a row a lane took 15 us
        // more for one tile)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          uint32_t pk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t lo, hi;
            f2_split(acc[4 * v + e], lo, hi);
            pk[e] = pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
          }
          sts128(box + lane * 256 + ((v ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
        }
        __syncwarp();
        const int rows = min(32, p.m - row0), cols = min(128, p.cols - col0);
        for (int r = 0; r < rows; ++r) {
          uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + static_cast<int64_t>(row0 + r) * p.cols + col0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = 64 * h + 2 * lane;
            const uint32_t w = lds32(box + r * 256 + (((col >> 3) ^ (r & 7)) << 4) + 2 * (col & 7));
            if (col + 1 < cols && p.cols % 2 == 0) {
              *reinterpret_cast<uint32_t*>(y + col) = w;
            } else {
              if (col < cols) y[col] = static_cast<uint16_t>(w);
              if (col + 1 < cols) y[col + 1] = static_cast<uint16_t>(w >> 16);
            }
          }
        }
        __syncwarp();                          // the box is read before the next tile fills it
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

template <bool W_MN>
int launch(const CUtensorMap& x, const CUtensorMap& w, const CUtensorMap& o, const Fp8Gemm& p, int pairs,
           cudaStream_t st) {
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  const unsigned grid = 2 * static_cast<unsigned>(std::min<int64_t>(tiles, pairs));
  return host::launch_pdl(k_fp8_pair<W_MN>, dim3(grid), dim3(kFp8PairThreads), kFp8PairSmem, st, 2, x, w, o, p);
}

}  // namespace

int launch_fp8_pair(bool w_mn, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const CUtensorMap& tm_out,
                    const Fp8Gemm& p, int pairs, cudaStream_t st) {
  return w_mn ? launch<true>(tm_x, tm_w, tm_out, p, pairs, st) : launch<false>(tm_x, tm_w, tm_out, p, pairs, st);
}

cudaError_t set_fp8_pair_attributes() {
  const cudaError_t e =
      cudaFuncSetAttribute(k_fp8_pair<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFp8PairSmem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_fp8_pair<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFp8PairSmem);
}

}  // namespace qlora
