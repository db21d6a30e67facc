// glu_wide.cu -- the gated feed-forward block in BF16 on a 512 x 256 pair tile: each CTA owns 256 rows of
// the tile as two 128-row M-waves, whose FP32 accumulators fill all 512 TMEM columns side by side.
//
// Per stage of 64 of the summed dimension a CTA loads 256 rows of A (32 KB) and its half of B (16 KB) for 2 x 128 x 256
// x 64 multiply-adds, where the 256 x 256 tile (glu.cu) moves 64 KB: a quarter less L2 traffic per operation, which
// under the power cap also buys clock. There is no second accumulator: the epilogue first takes a wave's 128 columns a
// thread into registers, gives TMEM back, and only then applies the activation and stores, while the next tile's MMAs
// run. Eight epilogue warps, two per TMEM lane quadrant, each for half of a wave's features;
// the producer warpgroup gives up registers to them (setmaxnreg). Every operand lies in shared memory as boxes of 64 x
// 64 elements, whichever of its dimensions is innermost.
// Measured on GB300: 4000 x 14336 x 4096 535 us in a long run under the power cap (1.76 PFLOP/s), 486 in a short one;
// Three stages and a second store
// buffer for each epilogue warp took the same time as four stages and one.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "common.cuh"
#include "glu_act.cuh"
#include "glu_common.cuh"
#include "host_common.h"

namespace dtcp {
namespace {

__global__ void __launch_bounds__(PairWideLayout::NUM_THREADS, 1)
    glu_wide_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ GluParams p) {
  using L = PairWideLayout;
  pair_wide_cta<kPairGated>(maps, p, [&](const PairCta& c) {
    const uint32_t bar_tfull = c.base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 8 * L::WAVES;
    const uint32_t q = c.warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
    const uint32_t epi = c.warp - L::EPI_WARP0;
    const int h = static_cast<int>(epi >> 2);  // its half of a wave's features
    const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
    const int rows = p.main.rows, cols = p.main.cols;
    PairStaging st{c.base + L::OFF_EPI + epi * L::EPI_BYTES, 0u, p.save != 0};
    bool ok = true;
    PairItem item;
    for (int it = 0; ok && pair_item(p, c.cluster_idx, c.num_clusters, it, item); ++it) {
      const int columns = item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;  // of the item's accumulators
      const int width = columns / 4;                                     // features of this warp: 64 or 32
      const int col0 = item.n_blk * L::FEATURES + (item.half > 0 ? 2 * width : 0) + h * width;
#pragma unroll 1
      for (int w = 0; w < L::WAVES; ++w) {
        const int row0 =
            item.m_blk * L::TILE_M + static_cast<int>(c.rank) * L::CTA_M + w * 128 + static_cast<int>(q) * 32;
        const bool live = row0 < rows && col0 < cols;
        if (!__all_sync(0xffffffffu, wait_phase_inline(bar_tfull + 8 * w, static_cast<uint32_t>(it) & 1u, c.wctx,
                                                       status_code(kRoleEpilogue, w)))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t taddr = c.tmem_base + ((q * 32u) << 16) + static_cast<uint32_t>(w) * L::ACC_COLS +
                               static_cast<uint32_t>(h * width);
        uint32_t v[4][32];  // g, u of 32 features, g, u of the next 32
        if (live) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((k >> 1) * 32 < width) tmem_ld_32x32b_x32(taddr + (k >> 1) * 32 + (k & 1) * (columns / 2), v[k]);
          tmem_ld_wait();
        }
        // the wave's columns are read: hand them back to the MMA issuer (leader's barrier)
        tc_fence_before_sync();
        __syncwarp();
        if (c.lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * w);  // orders tcgen05 work only
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int col = col0 + k * 32;
          if (k * 32 < width && col < cols) {
            if (p.save) {
              pair_store(st, c.lane, &maps.c1, v[2 * k], col, row0, true, kPairStreaming);
              pair_store(st, c.lane, &maps.c2, v[2 * k + 1], col, row0, true, kPairStreaming);
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              v[2 * k][j] = __float_as_uint(glu_act(__uint_as_float(v[2 * k][j]), p.act) *
                                            __uint_as_float(v[2 * k + 1][j]));
            pair_store(st, c.lane, &maps.c0, v[2 * k], col, row0, false);
          }
        }
      }
    }
    if (c.lane == 0) bulk_wait_group<0>();
    __syncwarp();
  });
}

}  // namespace

// ---------------------------------------------------------------- host side

int glu_wide_max_clusters(int device) {
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (cache[device] == 0) {
    const void* kernel = reinterpret_cast<const void*>(glu_wide_kernel);
    cache[device] = pair_max_clusters(&kernel, 1, true);
  }
  return cache[device];
}

int glu_wide_launch(const PairMaps& m, const GluParams& p, int clusters, cudaStream_t stream) {
  void* args[] = {const_cast<PairMaps*>(&m), const_cast<GluParams*>(&p)};
  return pair_launch(reinterpret_cast<const void*>(glu_wide_kernel), args, true, clusters, stream);
}

}  // namespace dtcp
