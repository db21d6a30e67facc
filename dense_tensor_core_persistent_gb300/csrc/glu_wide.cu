// glu_wide.cu -- the BF16 products of the gated feed-forward block on a 512 x 256 pair tile: each CTA owns 256 rows of
// the tile as two 128-row M-waves, whose FP32 accumulators fill all 512 TMEM columns side by side.
//
// Per stage of 64 of the summed dimension a CTA loads 256 rows of A (32 KB) and its half of B (16 KB) for 2 x 128 x 256
// x 64 multiply-adds, where the 256 x 256 tile (glu.cu) moves 64 KB: a quarter less L2 traffic per operation, which
// under the power cap also buys clock. There is no second accumulator: the epilogue first takes a wave's 128 columns a
// thread into registers, gives TMEM back, and only then applies the activation and stores, while the next tile's MMAs
// run. Eight epilogue warps, two per TMEM lane quadrant, each for half of a wave's columns (forward: of its features);
// the producer warpgroup gives up registers to them (setmaxnreg). Every operand lies in shared memory as boxes of 64 x
// 64 elements, whichever of its dimensions is innermost.
// Measured on GB300: 4000 x 14336 x 4096 535 us in a long run under the power cap (1.76 PFLOP/s), 486 in a short one;
// the gradient's products at 4096 x 14336 x 4096 962 to 1002 us (1.9 to 2.0 PFLOP/s). Three stages and a second store
// buffer for each epilogue warp took the same time as four stages and one.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "glu_act.cuh"
#include "glu_common.cuh"
#include "host_common.h"

namespace dtcp {

struct GluWideLayout {
  static constexpr int CG = 2, WAVES = 2;
  static constexpr int CTA_M = 256, TILE_M = 512;
  static constexpr int BLOCK_N = 256, FEATURES = 128;
  static constexpr int STAGE_K = 64, KSTEPS = 4, STAGES = 4;
  static constexpr int BOX_BYTES = 64 * 128;          // 64 x 64 BF16
  static constexpr int WAVE_BYTES = 2 * BOX_BYTES;    // 128 rows of A
  static constexpr int A_BOXES = 4, B_BOXES = 2;
  static constexpr int A_BYTES = A_BOXES * BOX_BYTES, B_BYTES = B_BOXES * BOX_BYTES;
  static constexpr int ACC_COLS = 256, TMEM_COLS = 512;
  static constexpr int WARP_A = 0, WARP_MMA = 1, WARP_B = 2, EPI_WARP0 = 4, EPI_WARPS = 8;
  static constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  // registers per thread after setmaxnreg (the launch gives 65536 / 384 -> 168)
  static constexpr int REGS_LAUNCH = 168, REGS_LOW = 56, REGS_EPI = 216;
  static constexpr int EPI_BYTES = kGluStagingBytes;
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_EPI = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + EPI_WARPS * EPI_BYTES;
  // full[S], empty[S], tmem_full[WAVES], tmem_empty[WAVES], drain
  static constexpr int NUM_BARS = 2 * STAGES + 2 * WAVES + 1;
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;  // slack to align the base to 1024 bytes
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(OFF_EPI % 1024 == 0, "1024-byte alignment");
  static_assert(NUM_THREADS * REGS_LAUNCH <= 65536 && 128 * REGS_LOW + 256 * REGS_EPI <= NUM_THREADS * REGS_LAUNCH,
                "setmaxnreg split exceeds the block's launch registers");
};

namespace {

// ---------------------------------------------------------------- producers (warps 0, 2)

template <bool BACKWARD>
__device__ __forceinline__ void glu_wide_producer(const GluParams& p, const GluMaps& maps, uint32_t base, uint32_t rank,
                                                  bool load_a, int cluster_idx, int num_clusters, const WaitCtx& wctx) {
  using L = GluWideLayout;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t dst0 = base + (load_a ? L::OFF_A : L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  GluItem item;
  for (int it = 0; ok && glu_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const int half = item.half > 0 ? 1 : 0;
    const int b_boxes = item.half >= 0 ? 1 : L::B_BOXES;
    const uint32_t stage_bytes = L::A_BYTES + static_cast<uint32_t>(b_boxes) * L::BOX_BYTES;
    const bool down = (it & 1) != 0;  // start on the blocks the last wave of tiles read last
    const int k_iters = item.second ? p.second.k_iters : p.main.k_iters;
    const CUtensorMap *m0, *m1;  // of the first and the second half of the stages
    int first;                   // the operand's first row (K-major) or column (MN-major)
    bool mn;
    if (load_a) {
      int mb = item.m_blk;
      m0 = &maps.a0;
      m1 = &maps.a1;
      if (BACKWARD && item.second && mb >= p.second.num_m_blocks / 2) {
        mb -= p.second.num_m_blocks / 2;
        m0 = m1;
      }
      first = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M;
      mn = BACKWARD && item.second;
    } else if (!BACKWARD) {
      m0 = m1 = rank == 1 ? &maps.b1 : &maps.b0;
      first = item.n_blk * L::FEATURES + half * (L::FEATURES / 2);
      mn = false;
    } else {
      m0 = item.second ? &maps.b2 : &maps.b0;
      m1 = &maps.b1;
      first = item.n_blk * L::BLOCK_N + half * (L::BLOCK_N / 2) + static_cast<int>(rank) * 64 * b_boxes;
      mn = true;
    }
    const int half_iters = BACKWARD && !item.second ? k_iters / 2 : k_iters;
    const int boxes = load_a ? L::A_BOXES : b_boxes;
    const uint32_t stride = load_a ? L::A_BYTES : L::B_BYTES;
    for (int kb = 0; kb < k_iters; ++kb) {
      if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
        ok = false;
        break;
      }
      int k = down ? k_iters - 1 - kb : kb;
      const CUtensorMap* map = m0;
      if (k >= half_iters) {
        k -= half_iters;
        map = m1;
      }
      const uint32_t full = bar_full + 8 * stage;
      if (load_a && rank == 0) mbar_arrive_expect_tx(full, 2u * stage_bytes);
      const uint32_t bar = mapa_shared(full, 0);
      const uint32_t dst = dst0 + stage * stride;
      for (int i = 0; i < boxes; ++i) {
        const int x = mn ? first + i * 64 : k * L::STAGE_K, y = mn ? k * L::STAGE_K : first + i * 64;
        tma_load_2d_pair(dst + i * L::BOX_BYTES, map, x, y, bar);
      }
      stage = stage + 1 == L::STAGES ? 0u : stage + 1;
      phase = stage == 0 ? phase ^ 1u : phase;
    }
  }
  if (!ok) settle_after_abort();
}

// ---------------------------------------------------------------- MMA issuer (leader, warp 1)

template <bool BACKWARD>
__device__ __forceinline__ void glu_wide_mma(const GluParams& p, uint32_t base, uint32_t tmem_base, int cluster_idx,
                                             int num_clusters, const WaitCtx& wctx) {
  using L = GluWideLayout;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 8 * L::WAVES;
  const uint32_t bar_drain = bar_tempty + 8 * L::WAVES;
  const uint64_t a_k = umma_desc_sw128(base + L::OFF_A), a_mn = umma_desc_mn(base + L::OFF_A, L::BOX_BYTES);
  const uint64_t b0 = BACKWARD ? umma_desc_mn(base + L::OFF_B, L::BOX_BYTES) : umma_desc_sw128(base + L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  GluItem item;
  for (int it = 0; ok && glu_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const bool dw = BACKWARD && item.second;
    const uint32_t idesc = idesc_glu(256, item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N, dw, BACKWARD);
    const bool down = (it & 1) != 0;
    const uint32_t free_parity = (static_cast<uint32_t>(it) & 1u) ^ 1u;
    const GluProduct& q = item.second ? p.second : p.main;
    const int half_iters = BACKWARD && !item.second ? q.k_iters / 2 : q.k_iters;
    for (int kb = 0; kb < q.k_iters; ++kb) {
      if (kb == 0 && !wait_phase_inline(bar_tempty, free_parity, wctx, status_code(kRoleMma, 0x100))) {
        ok = false;
        break;
      }
      if (!wait_phase_inline(bar_full + 8 * stage, phase, wctx, status_code(kRoleMma, stage))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      int k = down ? q.k_iters - 1 - kb : kb;
      if (k >= half_iters) k -= half_iters;
      const int left = q.depth - k * L::STAGE_K;  // a ragged last stage: only the MMAs that hold any of it
      const int steps = left >= L::STAGE_K ? L::KSTEPS : (left + 15) / 16;
      const uint64_t b = umma_desc_advance(b0, stage * L::B_BYTES);
      auto wave = [&](int w) {
        const uint32_t d = tmem_base + static_cast<uint32_t>(w) * L::ACC_COLS;
        const uint32_t offset = stage * L::A_BYTES + static_cast<uint32_t>(w) * L::WAVE_BYTES;
        const uint64_t a = umma_desc_advance(dw ? a_mn : a_k, offset);
        auto one = [&](int kk) {
          const uint32_t step_k = static_cast<uint32_t>(kk) * 32u, step_mn = static_cast<uint32_t>(kk) * 2048u;
          mma_f16<2>(d, umma_desc_advance(a, dw ? step_mn : step_k),
                     umma_desc_advance(b, BACKWARD ? step_mn : step_k), idesc, (kb | kk) != 0 ? 1u : 0u);
        };
        if (steps == L::KSTEPS) {
#pragma unroll
          for (int kk = 0; kk < L::KSTEPS; ++kk) one(kk);
        } else {
          for (int kk = 0; kk < steps; ++kk) one(kk);
        }
      };
      wave(0);
      if (kb + 1 == q.k_iters) mma_commit_pair_multicast(bar_tfull, 0x3);
      if (kb == 0) {
        if (!wait_phase_inline(bar_tempty + 8, free_parity, wctx, status_code(kRoleMma, 0x101))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
      }
      wave(1);
      if (kb + 1 == q.k_iters) mma_commit_pair_multicast(bar_tfull + 8, 0x3);
      mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
      stage = stage + 1 == L::STAGES ? 0u : stage + 1;
      phase = stage == 0 ? phase ^ 1u : phase;
    }
  }
  if (!ok) {
    // let issued MMAs finish before TMEM is released (bounded: they finish or the limit passes)
    mma_commit_pair_multicast(bar_drain, 0x1);
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_suspend(bar_drain, 0, 20000u) && globaltimer_ns() - t0 < wctx.limit_ns) {
    }
    settle_after_abort();
  }
}

// ---------------------------------------------------------------- epilogue (warps 4..11)

template <bool BACKWARD>
__device__ __forceinline__ void glu_wide_epilogue(const GluParams& p, const GluMaps& maps, uint32_t base,
                                                  uint32_t tmem_base, uint32_t warp, uint32_t lane, uint32_t rank,
                                                  int cluster_idx, int num_clusters, const WaitCtx& wctx) {
  using L = GluWideLayout;
  const uint32_t bar_tfull = base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 8 * L::WAVES;
  const uint32_t q = warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
  const uint32_t epi = warp - L::EPI_WARP0;
  const int h = static_cast<int>(epi >> 2);  // its half of a wave's columns
  const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
  GluStaging st{base + L::OFF_EPI + epi * L::EPI_BYTES, 0u, !BACKWARD && p.save != 0};
  bool ok = true;
  GluItem item;
  for (int it = 0; ok && glu_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const int columns = item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;  // of the item's accumulators
    const int width = columns / (BACKWARD ? 2 : 4);  // output columns of this warp: 128 or 64; forward 64 or 32
    const int col0 = item.n_blk * (BACKWARD ? L::BLOCK_N : L::FEATURES) + (item.half > 0 ? 2 * width : 0) + h * width;
    int mb = item.m_blk, rows = p.main.rows, cols = p.main.cols;
    const CUtensorMap* out = &maps.c0;
    if (BACKWARD && item.second) {
      const int half_blocks = p.second.num_m_blocks / 2;
      out = mb >= half_blocks ? &maps.c2 : &maps.c1;
      if (mb >= half_blocks) mb -= half_blocks;
      rows = p.second.rows;
      cols = p.second.cols;
    }
#pragma unroll 1
    for (int w = 0; w < L::WAVES; ++w) {
      const int row0 = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M + w * 128 + static_cast<int>(q) * 32;
      const bool live = row0 < rows && col0 < cols;
      if (!__all_sync(0xffffffffu, wait_phase_inline(bar_tfull + 8 * w, static_cast<uint32_t>(it) & 1u, wctx,
                                                     status_code(kRoleEpilogue, w)))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t taddr = tmem_base + ((q * 32u) << 16) + static_cast<uint32_t>(w) * L::ACC_COLS +
                             static_cast<uint32_t>(h * width);
      // backward: four chunks of 32 columns; forward: g, u of 32 features, g, u of the next 32
      uint32_t v[4][32];
      if (live) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (BACKWARD) {
            if (c * 32 < width) tmem_ld_32x32b_x32(taddr + c * 32, v[c]);
          } else {
            if ((c >> 1) * 32 < width) tmem_ld_32x32b_x32(taddr + (c >> 1) * 32 + (c & 1) * (columns / 2), v[c]);
          }
        }
        tmem_ld_wait();
      }
      // the wave's columns are read: hand them back to the MMA issuer (leader's barrier)
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * w);  // orders tcgen05 work only
      if (!live) continue;
      if constexpr (BACKWARD) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 32 < width && col0 + c * 32 < cols) glu_store(st, lane, out, v[c], col0 + c * 32, row0, false);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = col0 + c * 32;
          if (c * 32 < width && col < cols) {
            if (p.save) {
              glu_store(st, lane, &maps.c1, v[2 * c], col, row0, true);
              glu_store(st, lane, &maps.c2, v[2 * c + 1], col, row0, true);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[2 * c][j] = __float_as_uint(glu_act(__uint_as_float(v[2 * c][j]), p.act) *
                                            __uint_as_float(v[2 * c + 1][j]));
            glu_store(st, lane, out, v[2 * c], col, row0, false);
          }
        }
      }
    }
  }
  if (lane == 0) bulk_wait_group<0>();
  __syncwarp();
}

// All roles meet here once their work is done; the MMA warp (which allocated TMEM) frees it.
__device__ __forceinline__ void glu_wide_teardown(uint32_t warp, uint32_t tmem_base) {
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == GluWideLayout::WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem_base, GluWideLayout::TMEM_COLS);
  }
}

template <bool BACKWARD>
__global__ void __launch_bounds__(GluWideLayout::NUM_THREADS, 1)
    glu_wide_kernel(const __grid_constant__ GluMaps maps, const __grid_constant__ GluParams p) {
  using L = GluWideLayout;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // same offset in both CTAs of a pair
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster_idx = static_cast<int>(blockIdx.x) / L::CG, num_clusters = static_cast<int>(gridDim.x) / L::CG;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 8 * L::WAVES;
  const uint32_t bar_drain = bar_tempty + 8 * L::WAVES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_TMEM_SLOT);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_ABORT);
  const WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int w = 0; w < L::WAVES; ++w) {
      mbar_init(bar_tfull + 8 * w, 1);
      mbar_init(bar_tempty + 8 * w, L::EPI_WARPS * L::CG);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0u;
    fence_mbarrier_init_cluster();
  }
  if (warp == L::WARP_MMA) {
    tmem_alloc<2>(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish<2>();
  }
  tc_fence_before_sync();
  cluster_sync_all();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();

  // One branch per role group, each running to the end of the kernel (the code after a change of register limit
  // belongs to that limit).
  if (warp < L::EPI_WARP0) {
    regs_decrease<L::REGS_LOW>();
    if (lane == 0) {
      if (warp == L::WARP_A || warp == L::WARP_B)
        glu_wide_producer<BACKWARD>(p, maps, base, rank, warp == L::WARP_A, cluster_idx, num_clusters, wctx);
      else if (warp == L::WARP_MMA && rank == 0)
        glu_wide_mma<BACKWARD>(p, base, tmem_base, cluster_idx, num_clusters, wctx);
    }
    __syncwarp();
    glu_wide_teardown(warp, tmem_base);
  } else {
    regs_increase<L::REGS_EPI>();
    glu_wide_epilogue<BACKWARD>(p, maps, base, tmem_base, warp, lane, rank, cluster_idx, num_clusters, wctx);
    glu_wide_teardown(warp, tmem_base);
  }
}

}  // namespace

// ---------------------------------------------------------------- host side

int glu_wide_max_clusters(int device) {
  using L = GluWideLayout;
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (cache[device] > 0) return cache[device];
  for (auto k : {glu_wide_kernel<false>, glu_wide_kernel<true>})
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_BYTES) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(2 * 16, 1, 1);
  cfg.blockDim = dim3(L::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = L::SMEM_BYTES;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = L::CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, glu_wide_kernel<false>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  cache[device] = n;
  return n;
}

int glu_wide_launch(const GluMaps& m, const GluParams& p, bool backward, int clusters, cudaStream_t stream) {
  using L = GluWideLayout;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * L::CG), 1, 1);
  cfg.blockDim = dim3(L::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = L::SMEM_BYTES;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = L::CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, backward ? glu_wide_kernel<true> : glu_wide_kernel<false>, m, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

}  // namespace dtcp
