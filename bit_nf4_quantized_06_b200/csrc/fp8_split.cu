// 8-bit product in 128 x 128 tiles with the reduction split over a cluster,
// sm_100a: the kernel of single tokens, batches and short inputs.
//
//   D[128 rows x 128 outputs] = sum_b (sx[row][b] sw[output block][b]) X_b[128 x 128] W_b[128 x 128]^T
//
// A few rows read the whole weight once, so the time is that of the weight's
// stream and of the latencies around it; what counts is that every SM takes
// part and keeps loads in flight. The CTAs of a cluster (up to eight) share
// one tile: each takes a range of the reduction blocks, keeps its fp32 sums in
// registers (the block's product comes from tensor memory and is added times
// its scales, as in the pair kernel; four buffers of 128 columns), leaves them
// in its shared memory, and after a cluster barrier every CTA adds up its
// share of the rows from all of them, in rank order, and writes bf16. One
// launch, no atomics, no scratch memory, results that repeat bit for bit.
//
// Up to kFp8QuantRows rows in bf16 (QUANT) are quantized here, by the scale warps,
// straight into the stages, in every CTA anew: one launch less for a single
// token, and no pass through memory (4096 x 4096 weight, 1 row: 10.1 us a call
// from Python and 7.2 on the device; with a launch of its own 15.1 and 7.5. More
// rows than a pass of the two warps holds made the device time longer: 16 rows
// 14.3 us).
//
// When the rows were quantized by the kernel launched right before, that
// kernel has itself waited for everything earlier: the weight's first stages
// are then requested before waiting for it (p.early_w).
//
// Measured (rows in 8 bits, device time): 4096 x 4096 weight, 1 row, S = 4: 6.0 us
// (2.8 TB/s of weight); 11008 x 4096, 37 rows, S = 1: 12.9 us (3.5 TB/s). Of that
// some 5 us pass before and after the stream (launch, barriers and tensor
// memory, the first load, joining and writing), and a reduction block costs a
// CTA some 450 cycles of epilogue, where the tensor core needs 256. Two groups of
// epilogue warps on alternate blocks made a block shorter (8 rows, 86 blocks in
// one CTA: 23.6 -> 24.9 with the longer end: no gain) and were not kept, nor were
// up to eleven narrower stages for few rows (the same time).
//
// Warps (384 threads): 0 TMA; 1 tensor-memory allocation and MMA issue; 2-3
// scales; 4-11 epilogue (lane quarter = warp % 4, output half = (warp - 4) / 4).
// Every wait is bounded.
#include <algorithm>

#include "fp8_gemm.cuh"
#include "host.h"

namespace qlora {
namespace {

using namespace tcd;

constexpr int kStages = 6;                     // 16 KB of rows and 16 KB of weight each
constexpr int kThreads = 384;
constexpr int kBufs = 4;
constexpr int kPartStride = 132;               // fp32 words of a row of partial sums
constexpr int kScaleChunk = 8, kScaleStride = 132;
constexpr int kQuantChunk = 4;                 // blocks of a chunk where the rows are quantized here: at once
constexpr int kRing = 2 * kScaleChunk * kScaleStride * 4;
constexpr int kSmem = kStages * 32768 + kRing + 1024 + 256;
static_assert(128 * kPartStride * 4 <= kStages * 32768, "partial sums reuse the stages");

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// grid: tiles x splits CTAs, clusters of `splits`; p.box_m rows a row box.
template <bool W_MN, bool QUANT>
__global__ void __launch_bounds__(kThreads, 1)
    k_fp8_split(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, Fp8Gemm p) {
  constexpr uint32_t HALF = 16384;
  constexpr uint32_t STAGE_BYTES = 2 * HALF;
  constexpr int CHUNK = QUANT ? kQuantChunk : kScaleChunk;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t ring = base + kStages * STAGE_BYTES;
  const uint32_t bar0 = ring + kRing;
  uint8_t* const ctl = smem_raw + (bar0 - raw);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto bar_accf = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
  auto bar_acce = [&](int b) { return bar0 + 8u * (2 * kStages + kBufs + b); };       // the live epilogue warps
  auto bar_sf = [&](int c) { return bar0 + 8u * (2 * kStages + 2 * kBufs + c); };      // two scale warps
  auto bar_se = [&](int c) { return bar0 + 8u * (2 * kStages + 2 * kBufs + 2 + c); };  // the live epilogue warps
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(ctl + 8 * (2 * kStages + 2 * kBufs + 4));
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const Fp8Abort ab{abort_flag, p.status};

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.splits;
  const int row0 = (tile % p.tiles_m) * 128, col0 = (tile / p.tiles_m) * 128;
  // this CTA's reduction blocks: as even a cut as blocks allow
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kblocks) * rank / p.splits);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kblocks) * (rank + 1) / p.splits);
  const int rows = min(128, p.m - row0);
  const int live = (rows + 31) >> 5;           // lane quarters with rows of their own; the others' warps take no part

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), QUANT ? 3 : 1);   // the producer, and the warps that write the rows
      mbar_init(bar_empty(s), 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(bar_accf(b), 1);
      mbar_init(bar_acce(b), 2 * live);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(bar_sf(c), 2);
      mbar_init(bar_se(c), 2 * live);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  grid_dependency_trigger();

  if (warp == 0) {
    if (lane == 0) {
      if (!QUANT) tma_prefetch_desc(&tm_x);
      tma_prefetch_desc(&tm_w);
      const uint32_t tx = HALF + (QUANT ? 0u : static_cast<uint32_t>(p.box_m) * 128);
      auto load_w = [&](int kb, int s) {
        mbar_arrive_expect_tx(bar_full(s), tx);
        const uint32_t dst = base + s * STAGE_BYTES + HALF;
        if (W_MN)
          tma_load_2d(dst, &tm_w, bar_full(s), col0, kb * 128);
        else
          tma_load_2d(dst, &tm_w, bar_full(s), kb * 128, col0);
      };
      const int n = kb1 - kb0, first = p.early_w ? min(n, kStages) : 0;
      for (int i = 0; i < first; ++i) load_w(kb0 + i, i);
      grid_dependency_wait();
      int it = 0;
      for (; it < n; ++it) {
        const int s = it % kStages;
        if (it >= first) {
          if (!fp8_wait(bar_empty(s), ((it / kStages) & 1) ^ 1, ab, QLORA_DEV_TIMEOUT_PRODUCER)) break;
          load_w(kb0 + it, s);
        }
        if (!QUANT) tma_load_2d(base + s * STAGE_BYTES, &tm_x, bar_full(s), (kb0 + it) * 128, row0);
      }
      // every load has landed once its stage's MMAs are done (or, given up on, at full)
      for (int j = max(0, it - kStages); j < it; ++j) drain_wait(bar_full(j % kStages), (j / kStages) & 1);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_fp8(128, 128, p.a_format, W_MN);
    const uint64_t dx0 = smem_desc_sw128(base, 16, 1024);
    const uint64_t dw0 = W_MN ? smem_desc_sw128(base + HALF, HALF, 1024) : smem_desc_sw128(base + HALF, 16, 1024);
    if (elect_one()) {
      int s = 0, b = 0, last = -1;
      uint32_t ph = 0, aph = 1, last_ph = 0;
      bool full = false, free = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!full && !fp8_wait(bar_full(s), ph, ab, QLORA_DEV_TIMEOUT_MMA)) break;
        if (!free && !fp8_wait(bar_acce(b), aph, ab, QLORA_DEV_TIMEOUT_MMA)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + b * 128, accf = bar_accf(b), empty = bar_empty(s);
        const uint64_t dx = dx0 + s * (STAGE_BYTES >> 4), dw = dw0 + s * (STAGE_BYTES >> 4);
        last = s;
        last_ph = ph;
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
        if (++b == kBufs) {
          b = 0;
          aph ^= 1;
        }
        full = fp8_token(bar_full(s), ph);
        free = fp8_token(bar_acce(b), aph);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_fp8(d, dx + kk * 2, dw + kk * (W_MN ? 256 : 2), idesc, kk > 0 ? 1u : 0u);
        tc_commit(accf);
        tc_commit(empty);
      }
      // the last stage issued is free: no MMA of this CTA is in flight any more
      if (last >= 0) drain_wait(bar_empty(last), last_ph);
    }
    __syncwarp();
  } else if (QUANT && warp < 4) {
    // row 2 (warp - 2) + lane / 16, eight values a lane, the blocks of a chunk at
    // once: one after the other their latencies made 1.2 us a block
    static_assert(kFp8QuantRows == 4, "two warps of two rows");
    grid_dependency_wait();
    const int l16 = lane & 15, r = 2 * (warp - 2) + (lane >> 4);
    const bool e5 = p.a_format == kE5M2;
    const float top = e5 ? fp8_top<kE5M2>() : fp8_top<kE4M3>();
    const int ob = col0 >> 7;
    uint4 v[CHUNK];
    float w = 0.0f;                            // lane i < CHUNK of warp 2: the weight's scale of block i
    auto request = [&](int k0) {
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        const int64_t col = static_cast<int64_t>(k0 + i) * 128 + 8 * l16;
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < rows && k0 + i < kb1 && col < p.red)      // p.red % 8 == 0
          v[i] = __ldg(reinterpret_cast<const uint4*>(p.x16 + r * p.red + col));
      }
      if (warp == 2 && lane < CHUNK && k0 + lane < kb1) w = __ldg(p.sw + ob * p.sw_out + (k0 + lane) * p.sw_red);
    };
    int c = 0, s = 0;
    uint32_t cph = 1, ph = 1;
    request(kb0);
    for (int k0 = kb0; k0 < kb1; k0 += CHUNK) {
      const int n = min(CHUNK, kb1 - k0);
      float a[CHUNK];
      uint32_t lo[CHUNK], hi[CHUNK];
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        a[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          a[i] = fmaxf(a[i], fmaxf(fp8_mag(__uint_as_float(u[j] << 16)), fp8_mag(__uint_as_float(u[j] & 0xFFFF0000u))));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < CHUNK; ++i) a[i] = fmaxf(a[i], __shfl_xor_sync(0xFFFFFFFFu, a[i], o));
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        a[i] = fmaxf(a[i], kFp8Least);
        const float inv = top / a[i];
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[2 * j] = fp8_scaled(__uint_as_float(u[j] << 16), inv);
          f[2 * j + 1] = fp8_scaled(__uint_as_float(u[j] & 0xFFFF0000u), inv);
        }
        lo[i] = e5 ? fp8_pack4<kE5M2>(f[0], f[1], f[2], f[3]) : fp8_pack4<kE4M3>(f[0], f[1], f[2], f[3]);
        hi[i] = e5 ? fp8_pack4<kE5M2>(f[4], f[5], f[6], f[7]) : fp8_pack4<kE4M3>(f[4], f[5], f[6], f[7]);
      }
      if (!fp8_token(bar_se(c), cph)) fp8_wait(bar_se(c), cph, ab, QLORA_DEV_TIMEOUT_PRODUCER);
      __syncwarp();
      const uint32_t slot = ring + c * (CHUNK * kScaleStride * 4);
      if (warp == 2 && lane < CHUNK) sts32(slot + lane * (kScaleStride * 4) + 4 * 128, __float_as_uint(w));
      request(k0 + CHUNK);
#pragma unroll
      for (int i = 0; i < CHUNK; ++i) {
        if (i >= n) break;
        if (!fp8_token(bar_empty(s), ph)) fp8_wait(bar_empty(s), ph, ab, QLORA_DEV_TIMEOUT_PRODUCER);
        __syncwarp();
        if (r < rows) {
          // the 128-byte swizzle that a tensor copy would have made
          const uint32_t at = base + s * STAGE_BYTES + r * 128 + (((l16 >> 1) ^ (r & 7)) << 4) + 8 * (l16 & 1);
          sts32(at, lo[i]);
          sts32(at + 4, hi[i]);
          if (l16 == 0) sts32(slot + i * (kScaleStride * 4) + 4 * r, __float_as_uint(a[i] / top));
        }
        fence_proxy_async_smem();              // the tensor core reads what was written here
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_full(s));
          if (i + 1 == n) mbar_arrive(bar_sf(c));
        }
        if (++s == kStages) {
          s = 0;
          ph ^= 1;
        }
      }
      c ^= 1;
      if (c == 0) cph ^= 1;
    }
  } else if (warp < 4) {
    // scales: as in the pair kernel, a chunk requested while the one before is at work
    grid_dependency_wait();
    const int half = warp - 2;
    const int kl = lane & 7, rl = lane >> 3;
    const int r0 = row0 + 64 * half + rl;
    const int ob = col0 >> 7;
    float v[16], w = 0.0f;
    auto request = [&](int k0) {
      const int kb = k0 + kl;
      const bool in = kb < kb1;
      const float* sx = p.sx + static_cast<int64_t>(r0) * p.xblk + kb;
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = (in && r0 + 4 * j < p.m) ? __ldg(sx + 4 * j * p.xblk) : 0.0f;
      w = (in && half == 0 && rl == 0) ? __ldg(p.sw + ob * p.sw_out + kb * p.sw_red) : 0.0f;
    };
    int c = 0;
    uint32_t cph = 1;
    request(kb0);
    for (int k0 = kb0; k0 < kb1; k0 += kScaleChunk) {
      const uint32_t slot = ring + (c * kScaleChunk + kl) * (kScaleStride * 4);
      if (!fp8_token(bar_se(c), cph)) fp8_wait(bar_se(c), cph, ab, QLORA_DEV_TIMEOUT_PRODUCER);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; ++j) sts32(slot + 4 * (64 * half + rl + 4 * j), __float_as_uint(v[j]));
      if (half == 0 && rl == 0) sts32(slot + 4 * 128, __float_as_uint(w));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sf(c));
      c ^= 1;
      if (c == 0) cph ^= 1;
      request(k0 + kScaleChunk);
    }
  } else if ((warp & 3) < live) {
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + 64 * half;
    const uint32_t ring_x = ring + 4 * (32 * quarter + lane), ring_w = ring + 4 * 128;
    uint64_t acc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0;
    int b = 0, c = 0, left = 0;
    uint32_t bph = 0, cph = 0, slot = 0;
    bool ready = false;              // token of bar_accf(b)
    // the factor of the next block, `more` of them to come
    auto next_scale = [&](int more) -> float {
      if (left == 0) {
        if (!fp8_token(bar_sf(c), cph)) fp8_wait(bar_sf(c), cph, ab, QLORA_DEV_TIMEOUT_EPI);
        __syncwarp();
        left = min(more, CHUNK);
        slot = c * (CHUNK * kScaleStride * 4);
      }
      const float s = __uint_as_float(lds32(ring_x + slot)) * __uint_as_float(lds32(ring_w + slot));
      slot += kScaleStride * 4;
      if (--left == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_se(c));
        c ^= 1;
        if (c == 0) cph ^= 1;
      }
      return s;
    };
    float s = next_scale(kb1 - kb0);
#pragma unroll 1
    for (int kb = kb1 - kb0; kb > 0; --kb) {
      const uint64_t s2 = f2(s, s);
      if (!ready) fp8_wait(bar_accf(b), bph, ab, QLORA_DEV_TIMEOUT_EPI);
      __syncwarp();
      tc_fence_after();
      const uint32_t t = tbase + b * 128, acce = bar_acce(b);
      if (++b == kBufs) {
        b = 0;
        bph ^= 1;
      }
      uint32_t ra[16], rb[16], rc[16], rd[16];
      tmem_ld_32x32b_x16(t, ra);
      tmem_ld_32x32b_x16(t + 16, rb);
      tmem_ld_32x32b_x16(t + 32, rc);
      tmem_ld_32x32b_x16(t + 48, rd);
      if (kb > 1) s = next_scale(kb - 1);      // while the sums are on their way
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce);
      ready = fp8_token(bar_accf(b), bph);
      promote16(acc, ra, s2);
      promote16(acc + 8, rb, s2);
      promote16(acc + 16, rc, s2);
      promote16(acc + 24, rd, s2);
    }
    // All of this CTA's MMAs are done and its loads consumed: the sums go
    // where the stages were.
    const int r = 32 * quarter + lane;
    if (r < rows) {
      const uint32_t dst = base + (r * kPartStride + 64 * half) * 4;
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        uint32_t v[4];
        f2_split(acc[i], v[0], v[1]);
        f2_split(acc[i + 1], v[2], v[3]);
        sts128(dst + 8 * i, v[0], v[1], v[2], v[3]);
      }
    }
  }

  // every CTA's sums are in place (and its loads and MMAs are over)
  __syncwarp();
  if (p.splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (*abort_flag == 0) {
    // rows of the tile in turn over the cluster's ranks and this CTA's warps
    const int live = min(128, p.cols - col0);
    for (int r = rank + p.splits * warp; r < rows; r += p.splits * (kThreads / 32)) {
      __nv_bfloat16* y = p.y + static_cast<int64_t>(row0 + r) * p.cols + col0;
      const uint32_t src = base + r * kPartStride * 4 + 16 * lane;
      // this lane's four columns; also where they are then stored one by one (333
      // rows x 1003 x 4112: 11.4 us, with a remote load a column 13.3)
      auto sum = [&]() {
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int q = 0; q < p.splits; ++q) {
          const float4 v = ld_cluster_f4(p.splits > 1 ? mapa_shared(src, q) : src);
          t.x += v.x;
          t.y += v.y;
          t.z += v.z;
          t.w += v.w;
        }
        return make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
      };
      const int n = live - 4 * lane;
      if (n <= 0) continue;
      if (p.tma_out) {                        // cols % 8 == 0
        *reinterpret_cast<uint2*>(y + 4 * lane) = sum();
      } else {
        uint16_t* o = reinterpret_cast<uint16_t*>(y) + 4 * lane;
        const uint2 t = sum();
        o[0] = static_cast<uint16_t>(t.x);
        if (n > 1) o[1] = static_cast<uint16_t>(t.x >> 16);
        if (n > 2) o[2] = static_cast<uint16_t>(t.y);
        if (n > 3) o[3] = static_cast<uint16_t>(t.y >> 16);
      }
    }
  }
  tc_fence_before();
  if (p.splits > 1)
    cluster_sync_all();   // no CTA leaves while another reads its sums
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

template <bool W_MN, bool QUANT>
int launch(const CUtensorMap& x, const CUtensorMap& w, const Fp8Gemm& p, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(p.tiles_m) * static_cast<unsigned>(p.tiles_n) * p.splits;
  return host::launch_pdl(k_fp8_split<W_MN, QUANT>, dim3(grid), dim3(kThreads), kSmem, st, p.splits, x, w, p);
}

}  // namespace

int launch_fp8_split(bool w_mn, const CUtensorMap& tm_x, const CUtensorMap& tm_w, const Fp8Gemm& p, cudaStream_t st) {
  if (p.x16 != nullptr) return w_mn ? launch<true, true>(tm_x, tm_w, p, st) : launch<false, true>(tm_x, tm_w, p, st);
  return w_mn ? launch<true, false>(tm_x, tm_w, p, st) : launch<false, false>(tm_x, tm_w, p, st);
}

namespace {
int g_clusters[64][kFp8MaxSplits + 1];   // written by the device check, under its lock
}

cudaError_t set_fp8_split_attributes(int dev) {
  const auto a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  cudaError_t e = cudaFuncSetAttribute(k_fp8_split<false, false>, a, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_fp8_split<true, false>, a, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_fp8_split<false, true>, a, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k_fp8_split<true, true>, a, kSmem);
  for (int s = 1; e == cudaSuccess && s <= kFp8MaxSplits; ++s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = s;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&g_clusters[dev][s], k_fp8_split<false, false>, &cfg);
  }
  return e;
}

int fp8_split_clusters(int dev, int splits) { return g_clusters[dev][splits]; }

}  // namespace qlora
