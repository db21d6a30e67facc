// glu.cu -- the gated feed-forward block H = act(X Wg^T) * (X Wu^T) on sm_103a tensor cores, its
// form with E4M3 operands and a scale per row, and its gradient.
//
//   g = X Wg^T, u = X Wu^T (M x N, FP32),  H = act(g) u
//   dg = dH u act'(g), du = dH act(g),  dX = dg Wg + du Wu,  dWg = dg^T X,  dWu = du^T X
//
// One persistent, warp-specialised kernel template computes all four products on a 256 x 256 tile
// per CTA pair (cta_group::2 MMAs, M = 256, N = 256, FP32 accumulators, two of them in TMEM):
//   forward: A = X and B = 128 rows of Wg (the pair's first CTA loads them) over 128 rows of Wu (the
//            second one), so columns 0..127 of the accumulator are g and columns 128..255 are u of the
//            same features, and the epilogue has both in one TMEM lane: both projections, the
//            activation and the product are one kernel, and X is read once for the two.
//   dX:      A = [dg | du], B = [Wg ; Wu], the sum over both halves of the features in one accumulator.
//   dWg/dWu: A = dg or du, B = X, summed over the rows of X.
// One launch computes all three: the tiles of dX, which are the longest, come first, and where their last wave leaves
// clusters free, those go ahead with as many tiles of dW as take the same time. Where dX has so few tiles that one
// would be the whole launch, their sums are cut into slices with FP32 partial sums that a last kernel adds in order.
// The gradient's products need operands along their other dimension (W by columns, dg and X by
// columns). The MMA takes them as they lie in memory: TMA boxes of 64 columns x 128 rows put the
// non-summed dimension innermost and the descriptors say so ("MN-major"), so nothing is transposed.
//
// A last wave of tiles at most half full runs as halves of its tiles (N = 128 MMAs).
// BF16 products with enough tiles run on a 512 x 256 pair tile instead (glu_wide.cu; glu_wide_rule).
// A stage holds 128 (BF16) or 256 (E4M3) of the summed dimension, 8 MMAs per barrier wait, 3 stages.
// Warp roles: 0 loads A, 2 loads B, 1 allocates TMEM and issues the MMAs (leader CTA), 4..11 epilogue, two to each
// TMEM lane quadrant with half of the columns each; stores go through swizzled staging tiles and TMA.
//
// Bound by the tensor cores; up to kGluRows rows, where the bytes of Wg and Wu are the bound, glu_rows.cu computes H^T.
// Measured on GB300 with this tile: 4000 x 14336 x 4096 553 us (535 on the 512 x 256 one), 128 x 28672 x 8192 in E4M3
// 85 (82 as H^T); the gradient's first step, which only moves bytes, 120 us at 4096 x 14336 (6.8 TB/s).
//
// For the gradient g and u are kept in FP32 (8 bytes per element and a tenth of the block's time at
// most): kept in BF16 they would add a rounding to dg and du next to the one their MMA operand needs.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "glu_act.cuh"
#include "glu_common.cuh"
#include "host_common.h"

namespace dtcp {

struct GluLayout {
  static constexpr int CG = 2;
  static constexpr int CTA_M = 128, TILE_M = 256;
  static constexpr int BLOCK_N = 256, B_ROWS = 128;  // B rows each CTA loads
  static constexpr int FEATURES = 128;               // forward: features of a tile
  static constexpr int ATOMS = 2;                    // 128-byte swizzle rows of the summed dimension per stage
  static constexpr int KSTEPS = 8;                   // MMAs per stage, 32 bytes of a K-major row each
  static constexpr int STAGES = 3;
  static constexpr int ATOM_BYTES = 128 * 128;       // 128 rows (or 128 K x 64 columns) of 128 bytes
  static constexpr int OPERAND_BYTES = ATOMS * ATOM_BYTES;
  static constexpr int STAGE_BYTES = 2 * OPERAND_BYTES;
  static constexpr int ACC_COLS = 256, TMEM_COLS = 512;
  static constexpr int WARP_A = 0, WARP_MMA = 1, WARP_B = 2, EPI_WARP0 = 4, EPI_WARPS = 8;
  static constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = STAGES * OPERAND_BYTES;
  static constexpr int OFF_EPI = OFF_B + STAGES * OPERAND_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + EPI_WARPS * kGluStagingBytes;
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;  // slack to align the base to 1024 bytes
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(OFF_EPI % 1024 == 0, "1024-byte alignment");
};

namespace {

// kind::f8f6f4, E4M3 x E4M3 -> FP32 (operand formats 0), both operands K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---------------------------------------------------------------- producers (warps 0, 2)

template <int MODE>
__device__ __forceinline__ void glu_producer(const GluParams& p, const GluMaps& maps, uint32_t base, uint32_t rank,
                                             bool load_a, int cluster_idx, int num_clusters, const WaitCtx& wctx) {
  using L = GluLayout;
  constexpr bool FORWARD = MODE != kGluBackward;
  constexpr int STAGE_K = MODE == kGluForwardE4m3 ? 256 : 128;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t dst0 = base + (load_a ? L::OFF_A : L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  GluItem item;
  for (int it = 0; ok && glu_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const int half = item.half > 0 ? 1 : 0;
    const int b_boxes = item.half >= 0 ? 1 : 2;  // of 64 rows (K-major: per atom) or 64 columns (MN-major)
    const uint32_t stage_bytes = L::OPERAND_BYTES + L::OPERAND_BYTES / 2 * b_boxes;
    const bool down = (it & 1) != 0;  // start on the blocks the last wave of tiles read last
    const int k_iters = item.second ? p.second.k_iters : p.main.k_iters;
    const CUtensorMap *m0, *m1;  // of the first and the second half of the stages
    int first;                   // the operand's first row (K-major) or column (MN-major)
    bool mn;
    if (load_a) {
      int mb = item.m_blk;
      m0 = &maps.a0;
      m1 = &maps.a1;
      if (item.second) {
        const int half_blocks = p.second.num_m_blocks / 2;
        if (mb >= half_blocks) {
          mb -= half_blocks;
          m0 = m1;
        }
      }
      first = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M;
      mn = !FORWARD && item.second;
    } else if (FORWARD) {
      m0 = m1 = rank == 1 ? &maps.b1 : &maps.b0;
      first = item.n_blk * L::FEATURES + half * (L::FEATURES / 2);
      mn = false;
    } else {
      m0 = item.second ? &maps.b2 : &maps.b0;
      m1 = &maps.b1;
      first = item.n_blk * L::BLOCK_N + half * (L::BLOCK_N / 2) + static_cast<int>(rank) * 64 * b_boxes;
      mn = true;
    }
    const int half_iters = !FORWARD && !item.second ? k_iters / 2 : k_iters;
    for (int kb = 0; kb < item.k1 - item.k0; ++kb) {
      if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
        ok = false;
        break;
      }
      int k = down ? item.k1 - 1 - kb : item.k0 + kb;
      const CUtensorMap* map = m0;
      if (k >= half_iters) {
        k -= half_iters;
        map = m1;
      }
      const uint32_t full = bar_full + 8 * stage;
      if (load_a && rank == 0) mbar_arrive_expect_tx(full, 2u * stage_bytes);
      const uint32_t bar = mapa_shared(full, 0);
      const uint32_t dst = dst0 + stage * L::OPERAND_BYTES;
      if (mn) {
        const int boxes = load_a ? 2 : b_boxes;
        for (int c = 0; c < boxes; ++c)
          tma_load_2d_pair(dst + c * L::ATOM_BYTES, map, first + c * 64, k * STAGE_K, bar);
      } else {
#pragma unroll
        for (int a = 0; a < L::ATOMS; ++a) {
          const int x = k * STAGE_K + a * (STAGE_K / L::ATOMS);
          if (load_a) {
            tma_load_2d_pair(dst + a * L::ATOM_BYTES, map, x, first, bar);
          } else {
            for (int c = 0; c < b_boxes; ++c)
              tma_load_2d_pair(dst + a * L::ATOM_BYTES + c * (L::ATOM_BYTES / 2), map, x, first + c * 64, bar);
          }
        }
      }
      stage = stage + 1 == L::STAGES ? 0u : stage + 1;
      phase = stage == 0 ? phase ^ 1u : phase;
    }
  }
  if (!ok) settle_after_abort();
}

// ---------------------------------------------------------------- MMA issuer (leader, warp 1)

template <int MODE>
__device__ __forceinline__ void glu_mma(const GluParams& p, uint32_t base, uint32_t tmem_base, int cluster_idx,
                                        int num_clusters, const WaitCtx& wctx) {
  using L = GluLayout;
  constexpr bool FORWARD = MODE != kGluBackward, E4M3 = MODE == kGluForwardE4m3;
  constexpr int STAGE_K = E4M3 ? 256 : 128, MMA_K = E4M3 ? 32 : 16;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  const uint64_t a_k = umma_desc_sw128(base + L::OFF_A), a_mn = umma_desc_mn(base + L::OFF_A, L::ATOM_BYTES);
  const uint64_t b0 = FORWARD ? umma_desc_sw128(base + L::OFF_B) : umma_desc_mn(base + L::OFF_B, L::ATOM_BYTES);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  GluItem item;
  for (int it = 0; ok && glu_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const bool dw = !FORWARD && item.second;
    const uint32_t n = item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;
    const uint32_t idesc = E4M3 ? idesc_e4m3(256, n) : idesc_glu(256, n, dw, !FORWARD);
    const bool down = (it & 1) != 0;
    const uint32_t slot = static_cast<uint32_t>(it) & 1u;
    const GluProduct& q = item.second ? p.second : p.main;
    const int half_iters = !FORWARD && !item.second ? q.k_iters / 2 : q.k_iters;
    if (!wait_phase_inline(bar_tempty + 8 * slot, ((static_cast<uint32_t>(it) >> 1) & 1u) ^ 1u, wctx,
                           status_code(kRoleMma, 0x100 + slot))) {
      ok = false;
      break;
    }
    const uint32_t d = tmem_base + slot * L::ACC_COLS;
    for (int kb = 0; kb < item.k1 - item.k0; ++kb) {
      if (!wait_phase_inline(bar_full + 8 * stage, phase, wctx, status_code(kRoleMma, stage))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      int k = down ? item.k1 - 1 - kb : item.k0 + kb;
      if (k >= half_iters) k -= half_iters;
      const uint64_t a = umma_desc_advance(dw ? a_mn : a_k, stage * L::OPERAND_BYTES);
      const uint64_t b = umma_desc_advance(b0, stage * L::OPERAND_BYTES);
      const int left = q.depth - k * STAGE_K;  // a ragged last stage: only the MMAs that hold any of it
      const int steps = left >= STAGE_K ? L::KSTEPS : (left + MMA_K - 1) / MMA_K;
      // MMA kk of a stage: K-major operands advance 32 bytes inside the swizzle row, four per atom;
      // MN-major ones by 16 rows of 128 bytes.
      auto one = [&](int kk) {
        const uint32_t step_k = static_cast<uint32_t>((kk / 4) * L::ATOM_BYTES + (kk % 4) * 32);
        const uint32_t step_mn = static_cast<uint32_t>(kk) * 2048u;
        const uint64_t ad = umma_desc_advance(a, dw ? step_mn : step_k);
        const uint64_t bd = umma_desc_advance(b, FORWARD ? step_k : step_mn);
        if constexpr (E4M3) mma_e4m3_pair(d, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
        else mma_f16<2>(d, ad, bd, idesc, (kb | kk) != 0 ? 1u : 0u);
      };
      if (steps == L::KSTEPS) {
#pragma unroll
        for (int kk = 0; kk < L::KSTEPS; ++kk) one(kk);
      } else {
        for (int kk = 0; kk < steps; ++kk) one(kk);
      }
      mma_commit_pair_multicast(bar_empty + 8 * stage, 0x3);
      stage = stage + 1 == L::STAGES ? 0u : stage + 1;
      phase = stage == 0 ? phase ^ 1u : phase;
    }
    if (ok) mma_commit_pair_multicast(bar_tfull + 8 * slot, 0x3);
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

template <int MODE>
__device__ __forceinline__ void glu_epilogue(const GluParams& p, const GluMaps& maps, uint32_t base, uint32_t tmem_base,
                                             uint32_t warp, uint32_t lane, uint32_t rank, int cluster_idx,
                                             int num_clusters, const WaitCtx& wctx) {
  using L = GluLayout;
  constexpr bool FORWARD = MODE != kGluBackward;
  const uint32_t bar_tfull = base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 16;
  const uint32_t q = warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
  const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
  const uint32_t epi = warp - L::EPI_WARP0;
  const int h = static_cast<int>(epi >> 2);  // its half of the columns
  GluStaging st{base + L::OFF_EPI + epi * kGluStagingBytes, 0u, FORWARD ? p.save != 0 : p.main.slices > 1};
  GluItem item;
  for (int it = 0; glu_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const int columns = item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;  // of the item's accumulator
    const int width = columns / (FORWARD ? 4 : 2);  // output columns of this warp: forward 64 or 32, else 128 or 64
    const int col0 = item.n_blk * (FORWARD ? L::FEATURES : L::BLOCK_N) + (item.half > 0 ? 2 * width : 0) + h * width;
    const uint32_t slot = static_cast<uint32_t>(it) & 1u;
    int mb = item.m_blk, rows = p.main.rows, cols = p.main.cols;
    const CUtensorMap* out = &maps.c0;
    if (!FORWARD && item.second) {
      const int half_blocks = p.second.num_m_blocks / 2;
      out = mb >= half_blocks ? &maps.c2 : &maps.c1;
      if (mb >= half_blocks) mb -= half_blocks;
      rows = p.second.rows;
      cols = p.second.cols;
    }
    const int row0 = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M + static_cast<int>(q) * 32;
    // E4M3: this lane's row scale and its features' scales, while the MMAs run
    float x_scale = 1.0f, w_scale[2][L::FEATURES / 64];
    if constexpr (MODE == kGluForwardE4m3) {
      if (row0 + static_cast<int>(lane) < rows) x_scale = p.x_scale[row0 + lane];
#pragma unroll
      for (int c = 0; c < L::FEATURES / 64; ++c) {
        const int f = col0 + c * 32 + static_cast<int>(lane);
        w_scale[0][c] = f < cols ? p.g_scale[f] : 0.0f;
        w_scale[1][c] = f < cols ? p.u_scale[f] : 0.0f;
      }
    }
    if (!wait_phase_warp(bar_tfull + 8 * slot, (static_cast<uint32_t>(it) >> 1) & 1u, wctx,
                         status_code(kRoleEpilogue, slot)))
      break;
    tc_fence_after_sync();
    const uint32_t taddr = tmem_base + ((q * 32u) << 16) + slot * L::ACC_COLS + static_cast<uint32_t>(h * width);
    if (row0 < rows) {
      if constexpr (FORWARD) {
        const float xs = x_scale;
#pragma unroll MODE == kGluForwardE4m3 ? 2 : 1
        for (int c = 0; c < L::FEATURES / 2; c += 32) {
          const int col = col0 + c;
          if (c >= width || col >= cols) break;
          float gs = 0.0f, us = 0.0f;  // E4M3: the scales of feature col + lane
          if constexpr (MODE == kGluForwardE4m3) {
            gs = w_scale[0][c / 32];
            us = w_scale[1][c / 32];
          }
          uint32_t g[32], u[32];
          tmem_ld_32x32b_x32(taddr + c, g);
          tmem_ld_32x32b_x32(taddr + columns / 2 + c, u);
          tmem_ld_wait();
          if (p.save) {
            glu_store(st, lane, &maps.c1, g, col, row0, true);
            glu_store(st, lane, &maps.c2, u, col, row0, true);
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float gv = __uint_as_float(g[j]), uv = __uint_as_float(u[j]);
            if constexpr (MODE == kGluForwardE4m3) {
              gv *= xs * __shfl_sync(0xffffffffu, gs, j);
              uv *= xs * __shfl_sync(0xffffffffu, us, j);
            }
            g[j] = __float_as_uint(glu_act(gv, p.act) * uv);
          }
          glu_store(st, lane, out, g, col, row0, false);
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < width; c += 32) {
          const int col = col0 + c;
          if (col >= cols) break;
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c, v);
          tmem_ld_wait();
          const bool partial = p.main.slices > 1 && !item.second;
          glu_store(st, lane, out, v, col, row0 + item.slice * p.main.slice_rows, partial);
        }
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * slot);  // orders tcgen05 work only
  }
  if (lane == 0) bulk_wait_group<0>();
  __syncwarp();
}

template <int MODE>
__global__ void __launch_bounds__(GluLayout::NUM_THREADS, 1)
    glu_kernel(const __grid_constant__ GluMaps maps, const __grid_constant__ GluParams p) {
  using L = GluLayout;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // same offset in both CTAs of a pair
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cluster_idx = static_cast<int>(blockIdx.x) / L::CG, num_clusters = static_cast<int>(gridDim.x) / L::CG;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_TMEM_SLOT);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_ABORT);
  const WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_tfull + 8 * s, 1);
      mbar_init(bar_tempty + 8 * s, L::EPI_WARPS * L::CG);
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

  if (warp < L::EPI_WARP0) {
    if (lane == 0) {
      if (warp == L::WARP_A || warp == L::WARP_B)
        glu_producer<MODE>(p, maps, base, rank, warp == L::WARP_A, cluster_idx, num_clusters, wctx);
      else if (warp == L::WARP_MMA && rank == 0)
        glu_mma<MODE>(p, base, tmem_base, cluster_idx, num_clusters, wctx);
    }
    __syncwarp();
  } else {
    glu_epilogue<MODE>(p, maps, base, tmem_base, warp, lane, rank, cluster_idx, num_clusters, wctx);
  }
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == L::WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem_base, L::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- dg and du

// [dg | du] (M x 2N BF16) from dH and the kept g, u (M x 2N FP32): 8 columns per thread.
__global__ void __launch_bounds__(256) glu_gate_grad_kernel(const uint16_t* dh, long long lddh, const float* pre,
                                                            uint16_t* dgu, int N, long long vectors, int act) {
  pdl_launch_dependents();
  pdl_wait();
  const int per_row = N / 8;
  for (long long v = blockIdx.x * 256LL + threadIdx.x; v < vectors; v += gridDim.x * 256LL) {
    const long long row = v / per_row;
    const int col = static_cast<int>(v - row * per_row) * 8;
    const uint4 d4 = *reinterpret_cast<const uint4*>(dh + row * lddh + col);
    const float4* gp = reinterpret_cast<const float4*>(pre + row * 2 * N + col);
    const float4* up = reinterpret_cast<const float4*>(pre + row * 2 * N + N + col);
    // (read once: streaming loads)
    const float4 ga = __ldcs(gp), gb = __ldcs(gp + 1), ua = __ldcs(up), ub = __ldcs(up + 1);
    const float g[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
    const float u[8] = {ua.x, ua.y, ua.z, ua.w, ub.x, ub.y, ub.z, ub.w};
    const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float rg[2], ru[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float d = __uint_as_float(t == 0 ? dw[j] << 16 : dw[j] & 0xFFFF0000u);
        float a, da;
        glu_act_grad(g[2 * j + t], act, a, da);
        rg[t] = d * u[2 * j + t] * da;
        ru[t] = d * a;
      }
      og[j] = pack_bf16x2_rn(__float_as_uint(rg[0]), __float_as_uint(rg[1]));
      ou[j] = pack_bf16x2_rn(__float_as_uint(ru[0]), __float_as_uint(ru[1]));
    }
    *reinterpret_cast<uint4*>(dgu + row * 2 * N + col) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4*>(dgu + row * 2 * N + N + col) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

// ---------------------------------------------------------------- dX from its slices

// The sum of the slices' partial sums in their order, rounded once: 8 columns per thread.
__global__ void __launch_bounds__(128) glu_join_kernel(const float* partial, int slices, long long slice_size,
                                                       uint16_t* dx, long long lddx, int cols, long long vectors) {
  pdl_launch_dependents();
  pdl_wait();
  const long long v = blockIdx.x * 128LL + threadIdx.x;
  if (v >= vectors) return;
  const int per_row = cols / 8;
  const long long row = v / per_row;
  const int col = static_cast<int>(v - row * per_row) * 8;
  const float* at = partial + row * cols + col;
  float sum[8] = {};
#pragma unroll 4
  for (int s = 0; s < slices; ++s) {
    const float4 a = *reinterpret_cast<const float4*>(at + s * slice_size);
    const float4 b = *reinterpret_cast<const float4*>(at + s * slice_size + 4);
    const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += f[j];
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2_rn(__float_as_uint(sum[2 * j]), __float_as_uint(sum[2 * j + 1]));
  *reinterpret_cast<uint4*>(dx + row * lddx + col) = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------- host side

int glu_max_clusters(int device) {
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (cache[device] > 0) return cache[device];
  for (auto k : {glu_kernel<kGluForward>, glu_kernel<kGluForwardE4m3>, glu_kernel<kGluBackward>})
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, GluLayout::SMEM_BYTES) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(2 * 16, 1, 1);
  cfg.blockDim = dim3(GluLayout::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = GluLayout::SMEM_BYTES;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, glu_kernel<kGluForward>, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  cache[device] = n;
  return n;
}

// A BF16 operand in boxes of 64 elements of its rows (the summed dimension if it is K-major, else columns) x `rows`.
int map_in(CUtensorMap* m, const void* p, int cols, int rows, long long ld, int box_rows) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, rows, uint64_t(ld) * 2, 64, box_rows,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}
int map_out(CUtensorMap* m, const void* p, int cols, int rows, long long ld) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, rows, uint64_t(ld) * 2, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_64B);
}

// The tiles of a product; `rows` and `cols` are those of one output, of which `outputs` lie one after the other along
// the rows; tile_rows, cols_a_tile: rows of a pair's tile and output columns of its 256-column accumulator.
int plan_product(GluProduct* q, int rows, int cols, int depth, int stage, int halves, int outputs, int tile_rows,
                 int cols_a_tile) {
  q->rows = rows;
  q->cols = cols;
  q->depth = depth;
  q->k_iters = halves * ceil_div(depth, stage);
  const long long m = static_cast<long long>(outputs) * ceil_div(rows, tile_rows);
  q->num_n_blocks = ceil_div(cols, cols_a_tile);
  if (m * q->num_n_blocks > 0x1FFFFFFFLL) return GEMM_ERR_UNSUPPORTED_SHAPE;
  q->num_m_blocks = static_cast<int>(m);
  q->num_tiles = q->num_items = static_cast<int>(m * q->num_n_blocks);
  q->split_tiles = 0;
  q->slices = 1;
  return GEMM_OK;
}

// Parts of dX's summed dimension, where its few tiles would be the launch's longest path: the stages of a tile against
// the stages of all tiles of both products spread over the pairs (with two more for a short tile of dW's end). A part
// has 6 stages at least, the parts run at once, and what is saved has to pay for the partial sums and the kernel that
// adds them, some 4 us (8 stages). Measured on GB300, whole gradient: 512 x 4096 x 1024 44.2 us in one part and 24.3 in
// four, 300 x 1368 x 520 22.3 and 17.3 in three; 10 x 2072 x 5576, which stays whole, 30.2 and 33.0 in three.
int glu_slices(const GluProduct& dx, const GluProduct& dw, int wave) {
  const long long work = 1LL * dx.num_tiles * dx.k_iters + 1LL * dw.num_tiles * (dw.k_iters + 2);
  const int share = std::max<int>(6, static_cast<int>(std::min<long long>(work / wave, 0x7FFFFFFF)));
  const int slices = std::min({8, dx.k_iters / share, wave / dx.num_tiles});
  return slices > 1 && dx.k_iters - dx.k_iters / slices >= 12 ? slices : 1;
}

// The order of a product's tiles on `clusters` pairs, for operands of `bytes` per element.
void order_product(GluProduct* q, int clusters, int tile_rows, double bytes, long long l2_bytes) {
  constexpr int BLOCK_N = GluLayout::BLOCK_N;
  q->group_m = choose_group_m(static_cast<int>(std::min<long long>(1LL * q->num_m_blocks * tile_rows, 0x7FFFFFFF)),
                              static_cast<int>(std::min<long long>(1LL * q->num_n_blocks * BLOCK_N, 0x7FFFFFFF)),
                              std::max(q->depth, 1), tile_rows, BLOCK_N, bytes, 0.0, clusters, l2_bytes);
}

// The co-resident pairs take the tiles of both products (the second may have none).
template <int MODE>
int glu_launch(const GluMaps& m, GluParams& p, bool wide, double bytes, int device, const DeviceInfo* info,
               cudaStream_t stream) {
  using L = GluLayout;
  p.status = device_status_word(device);
  p.wait_limit_ns = RunOptions().wait_limit_ns;
  if (p.status == nullptr) return GEMM_ERR_NO_DEVICE;
  const int wave = wide ? glu_wide_max_clusters(device) : glu_max_clusters(device);
  if (wave <= 0) return GEMM_ERR_LAUNCH;
  GluProduct &a = p.main, &b = p.second;
  p.ahead = 0;
  if (b.num_tiles == 0 && a.slices == 1) {
    a.split_tiles = tail_split_tiles(a.num_tiles, wave);
    a.num_items = a.num_tiles + a.split_tiles;
  } else if (b.num_tiles > 0) {
    // clusters that a last partial wave of the first product leaves free go ahead with tiles of the second
    const int clusters = std::min(a.num_items + b.num_tiles, wave);
    const int in_last = a.num_items % clusters, idle = in_last > 0 ? clusters - in_last : 0;
    if (idle > 0)
      p.ahead = std::min((a.k_iters / a.slices + b.k_iters / 2) / b.k_iters, ceil_div(b.num_tiles, idle));
    const int rest = std::max(0, b.num_tiles - p.ahead * idle);
    b.split_tiles = tail_split_tiles(rest, wave);
    b.num_items = b.num_tiles + b.split_tiles;
  }
  const int clusters = std::min(a.num_items + b.num_items, wave);
  const int tile_rows = wide ? 2 * L::TILE_M : L::TILE_M;
  order_product(&a, clusters, tile_rows, bytes, info->l2_bytes);
  if (b.num_tiles > 0) order_product(&b, clusters, tile_rows, bytes, info->l2_bytes);
  if (wide) return glu_wide_launch(m, p, MODE == kGluBackward, clusters, stream);
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
  if (cudaLaunchKernelEx(&cfg, glu_kernel<MODE>, m, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// Whether BF16 products of the given tiles (512 rows each; std: 256 rows) and stages run on the 512 x 256 pair tile. It
// moves a quarter fewer bytes from L2 per operation but has half the tiles and one accumulator, so it needs a deep sum
// and is taken where the launch, in tile-times of the 256 x 256 tile, is shorter with wide tiles at 2 / 1.06 each:
// 1.06 is its gain per unit of work. Measured on GB300 on 64 shapes from 2048 deep on whose two estimates are within
// 12%: rows of X that start on 128-byte boundaries show 1.03 in the mean, forward (0.98 to 1.07: 178 us on the 256 x
// 256 tile and 174 on this one at 5951 x 3904 x 3264, 115 and 118 at 3853 x 5504 x 2176) and in the gradient (0.94 to
// 1.14); other rows 1.13 and 1.11 (352 and 300 us at 9034 x 5016 x 2744). The rule is 0.6% and 1.5% slower in the mean
// than the better tile of each shape on the former, 4% and 2% on the latter.
bool glu_wide_rule(long long std_tiles, long long wide_tiles, int depth, int wave) {
  return depth >= 2048 && 2.0 * launch_tile_times(wide_tiles, wave) / 1.06 < launch_tile_times(std_tiles, wave);
}

bool glu_forward_wide(int M, int N, int K, int wave) {
  using L = GluLayout;
  const long long n_tiles = ceil_div(N, L::FEATURES);
  return glu_wide_rule(ceil_div(M, L::TILE_M) * n_tiles, ceil_div(M, 2 * L::TILE_M) * n_tiles, K, wave);
}
bool glu_backward_wide(int M, int N, int K, bool dx, bool dw, int wave) {
  using L = GluLayout;
  if (M == 0) return false;
  // in tiles of dW (their depth is M), of which one of dX (depth 2 N) counts several
  const double long_tile = dw ? 2.0 * N / M : 1.0;
  const long long k_tiles = ceil_div(K, L::BLOCK_N);
  auto tiles = [&](int tile_rows) {
    return static_cast<long long>(dx ? long_tile * ceil_div(M, tile_rows) * k_tiles : 0.0) +
           (dw ? 2LL * ceil_div(N, tile_rows) * k_tiles : 0LL);
  };
  const int depth = !dw ? static_cast<int>(std::min(2LL * N, 0x7FFFFFFFLL)) : !dx ? M : std::min(M, N);
  return glu_wide_rule(tiles(L::TILE_M), tiles(2 * L::TILE_M), depth, wave);
}

bool known_act(int act) { return act == GEMM_GLU_SILU || act == GEMM_GLU_GELU_TANH || act == GEMM_GLU_RELU; }

int zero_rows(void* p, size_t row_bytes, long long ld_bytes, int rows, cudaStream_t s) {
  if (rows > 0 && row_bytes > 0 && cudaMemset2DAsync(p, ld_bytes, 0, row_bytes, rows, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

struct GluStrides {
  long long x, h, dh, dx;
};
// Strides in elements, 0 = contiguous; X's in multiples of 16 bytes.
int resolve_strides(const gemm_glu_strides_t* s, int N, int K, GluStrides* r) {
  *r = GluStrides{K, N, N, K};
  if (s == nullptr) return GEMM_OK;
  if (s->x) r->x = s->x;
  if (s->h) r->h = s->h;
  if (s->dh) r->dh = s->dh;
  if (s->dx) r->dx = s->dx;
  if (r->x < K || r->h < N || r->dh < N || r->dx < K) return GEMM_ERR_INVALID_ARG;
  return GEMM_OK;
}

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_glu_plan(int M, int N, int K, int wave, int* forward, int* backward) {
  if (M < 0 || N < 0 || K < 0 || wave <= 0 || forward == nullptr || backward == nullptr) return GEMM_ERR_INVALID_ARG;
  *forward = M <= kGluRows ? 0 : glu_forward_wide(M, N, K, wave) ? 512 : 256;
  *backward = glu_backward_wide(M, N, K, true, true, wave) ? 512 : 256;
  return GEMM_OK;
}

int gemm_glu_bf16(const void* X, const void* Wg, const void* Wu, void* H, float* preact, int M, int N, int K, int act,
                  void* stream, const gemm_glu_strides_t* strides) {
  using L = GluLayout;
  if (M < 0 || N < 0 || K < 0 || !known_act(act)) return GEMM_ERR_INVALID_ARG;
  GluStrides ld;
  if (resolve_strides(strides, N, K, &ld) != GEMM_OK) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  if (H == nullptr || (K > 0 && (X == nullptr || Wg == nullptr || Wu == nullptr))) return GEMM_ERR_INVALID_ARG;
  if (K % 8 != 0 || N % 8 != 0 || ld.x % 8 != 0 || ld.h % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(H) || !aligned16(preact) || (K > 0 && (!aligned16(X) || !aligned16(Wg) || !aligned16(Wu))))
    return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) {  // g = u = 0, and act(0) * 0 = 0
    int st = zero_rows(H, size_t(N) * 2, ld.h * 2, M, s);
    if (st == GEMM_OK && preact != nullptr) st = zero_rows(preact, size_t(N) * 8, (long long)N * 8, M, s);
    return st;
  }
  if (M <= kGluRows) {
    const GluRowsOperands f = {X,       Wg,   Wu,   static_cast<uint16_t*>(H), preact, nullptr, nullptr,
                               nullptr, ld.x, ld.h, M,                         N,      K,       act};
    return run_glu_rows(f, false, device, info, s);
  }
  GluMaps m;
  GluParams p = {};
  const bool wide = glu_forward_wide(M, N, K, glu_max_clusters(device));
  int st = map_in(&m.a0, X, K, M, ld.x, wide ? 64 : 128);
  if (st == GEMM_OK) st = map_in(&m.b0, Wg, K, N, K, 64);  // (half its rows: a half tile's load is one box)
  if (st == GEMM_OK) st = map_in(&m.b1, Wu, K, N, K, 64);
  if (st == GEMM_OK) st = map_out(&m.c0, H, N, M, ld.h);
  if (st != GEMM_OK) return st;
  m.a1 = m.b2 = m.a0;
  m.c1 = m.c2 = m.c0;
  if (preact != nullptr) {
    st = encode_tmap_2d(&m.c1, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, preact, N, M, uint64_t(N) * 8, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == GEMM_OK)
      st = encode_tmap_2d(&m.c2, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, preact + N, N, M, uint64_t(N) * 8, 32, 32,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != GEMM_OK) return st;
  }
  p.act = act;
  p.save = preact != nullptr ? 1 : 0;
  st = plan_product(&p.main, M, N, K, wide ? 64 : 128, 1, 1, wide ? 2 * L::TILE_M : L::TILE_M, L::FEATURES);
  return st != GEMM_OK ? st : glu_launch<kGluForward>(m, p, wide, 2.0, device, info, s);
}

int gemm_glu_e4m3(const void* X, const float* x_scale, const void* Wg, const float* wg_scale, const void* Wu,
                  const float* wu_scale, void* H, int M, int N, int K, int act, void* stream,
                  const gemm_glu_strides_t* strides) {
  using L = GluLayout;
  if (M < 0 || N < 0 || K < 0 || !known_act(act)) return GEMM_ERR_INVALID_ARG;
  GluStrides ld;
  if (resolve_strides(strides, N, K, &ld) != GEMM_OK) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  if (H == nullptr || (K > 0 && (X == nullptr || Wg == nullptr || Wu == nullptr || x_scale == nullptr ||
                                 wg_scale == nullptr || wu_scale == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 8 != 0 || ld.x % 16 != 0 || ld.h % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
  auto aligned4 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) == 0; };
  if (!aligned16(H) || (K > 0 && (!aligned16(X) || !aligned16(Wg) || !aligned16(Wu) || !aligned4(x_scale) ||
                                  !aligned4(wg_scale) || !aligned4(wu_scale))))
    return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return zero_rows(H, size_t(N) * 2, ld.h * 2, M, s);
  if (M <= kGluRows) {
    const GluRowsOperands f = {X,        Wg,   Wu,   static_cast<uint16_t*>(H), nullptr, x_scale, wg_scale,
                               wu_scale, ld.x, ld.h, M,                         N,       K,       act};
    return run_glu_rows(f, true, device, info, s);
  }
  GluMaps m;
  GluParams p = {};
  auto map8 = [&](CUtensorMap* t, const void* q, int rows, long long stride, int box_rows) {
    return encode_tmap_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, rows, stride, 128, box_rows,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  };
  int st = map8(&m.a0, X, M, ld.x, 128);
  if (st == GEMM_OK) st = map8(&m.b0, Wg, N, K, 64);
  if (st == GEMM_OK) st = map8(&m.b1, Wu, N, K, 64);
  if (st == GEMM_OK) st = map_out(&m.c0, H, N, M, ld.h);
  if (st != GEMM_OK) return st;
  m.a1 = m.b2 = m.a0;
  m.c1 = m.c2 = m.c0;
  p.act = act;
  p.x_scale = x_scale;
  p.g_scale = wg_scale;
  p.u_scale = wu_scale;
  st = plan_product(&p.main, M, N, K, 256, 1, 1, L::TILE_M, L::FEATURES);
  return st != GEMM_OK ? st : glu_launch<kGluForwardE4m3>(m, p, false, 1.0, device, info, s);
}

int gemm_glu_bf16_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const float* preact, void* dX,
                           void* dWg, void* dWu, int M, int N, int K, int act, void* stream,
                           const gemm_glu_strides_t* strides) {
  using L = GluLayout;
  if (M < 0 || N < 0 || K < 0 || !known_act(act)) return GEMM_ERR_INVALID_ARG;
  GluStrides ld;
  if (resolve_strides(strides, N, K, &ld) != GEMM_OK) return GEMM_ERR_INVALID_ARG;
  if ((dWg == nullptr) != (dWu == nullptr)) return GEMM_ERR_INVALID_ARG;
  const bool work = M > 0 && N > 0 && K > 0;
  if (work && (dX != nullptr || dWg != nullptr) &&
      (dH == nullptr || preact == nullptr || (dX != nullptr && (Wg == nullptr || Wu == nullptr)) ||
       (dWg != nullptr && X == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if (K % 8 != 0 || N % 8 != 0 || N > 0x3FFFFFFF || ld.x % 8 != 0 || ld.dh % 8 != 0 || ld.dx % 8 != 0)
    return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(dH) || !aligned16(X) || !aligned16(Wg) || !aligned16(Wu) || !aligned16(preact) || !aligned16(dX) ||
      !aligned16(dWg) || !aligned16(dWu))
    return GEMM_ERR_MISALIGNED;
  if ((dX == nullptr && dWg == nullptr) || K == 0 || (M == 0 && (dWg == nullptr || N == 0)) ||
      (N == 0 && (dX == nullptr || M == 0)))
    return GEMM_OK;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N == 0) return zero_rows(dX, size_t(K) * 2, ld.dx * 2, M, s);  // a sum over no features
  if (M == 0) {                                                      // sums over no rows
    int st = zero_rows(dWg, size_t(K) * 2, (long long)K * 2, N, s);
    return st != GEMM_OK ? st : zero_rows(dWu, size_t(K) * 2, (long long)K * 2, N, s);
  }
  GluParams p = {};
  p.main.slices = p.second.slices = 1;
  const int wave = glu_max_clusters(device);
  if (wave <= 0) return GEMM_ERR_LAUNCH;
  const bool wide = glu_backward_wide(M, N, K, dX != nullptr, dWg != nullptr, wave);
  const int stage = wide ? 64 : 128, tile_rows = wide ? 2 * L::TILE_M : L::TILE_M;
  int st = GEMM_OK;
  if (dX != nullptr) st = plan_product(&p.main, M, K, N, stage, 2, 1, tile_rows, L::BLOCK_N);
  if (st == GEMM_OK && dWg != nullptr) st = plan_product(&p.second, N, K, M, stage, 1, 2, tile_rows, L::BLOCK_N);
  if (st != GEMM_OK) return st;
  if (dX != nullptr && !wide) {
    p.main.slices = glu_slices(p.main, p.second, wave);
    p.main.num_items = p.main.num_tiles * p.main.slices;
    p.main.slice_rows = ceil_div(M, 32) * 32;
  }
  const int slices = p.main.slices;
  const size_t gate_bytes = size_t(M) * N * 4;  // N % 8 == 0: the partial sums start on a 16-byte boundary
  const size_t slice_size = slices > 1 ? size_t(p.main.slice_rows) * K : 0;
  cudaMemPool_t pool = workspace_pool(device);
  void* ws = nullptr;
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, gate_bytes + slices * slice_size * 4, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  float* const partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + gate_bytes);
  uint16_t* dgu = static_cast<uint16_t*>(ws);
  {
    const long long vectors = static_cast<long long>(M) * (N / 8);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>((vectors + 255) / 256, 8LL * info->num_sms)), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, glu_gate_grad_kernel, static_cast<const uint16_t*>(dH), ld.dh, preact, dgu, N, vectors,
                           act) != cudaSuccess) {
      cudaGetLastError();
      st = GEMM_ERR_LAUNCH;
    } else {
      count_launch();
      st = GEMM_OK;
    }
  }
  if (st == GEMM_OK) {
    GluMaps m;
    st = map_in(&m.a0, dgu, N, M, 2LL * N, stage);  // (a box of 64 features is the same for either order)
    if (st == GEMM_OK) st = map_in(&m.a1, dgu + N, N, M, 2LL * N, stage);
    m.b0 = m.b1 = m.b2 = m.c0 = m.c1 = m.c2 = m.a0;
    if (dX != nullptr) {
      if (st == GEMM_OK) st = map_in(&m.b0, Wg, K, N, K, stage);
      if (st == GEMM_OK) st = map_in(&m.b1, Wu, K, N, K, stage);
      if (st == GEMM_OK && slices == 1) st = map_out(&m.c0, dX, K, M, ld.dx);
      if (st == GEMM_OK && slices > 1)
        st = encode_tmap_2d(&m.c0, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, partial, K, uint64_t(slices) * p.main.slice_rows,
                            uint64_t(K) * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (dWg != nullptr) {
      if (st == GEMM_OK) st = map_in(&m.b2, X, K, M, ld.x, stage);
      if (st == GEMM_OK) st = map_out(&m.c1, dWg, K, N, K);
      if (st == GEMM_OK) st = map_out(&m.c2, dWu, K, N, K);
    }
    if (st == GEMM_OK) st = glu_launch<kGluBackward>(m, p, wide, 2.0, device, info, s);
    if (st == GEMM_OK && slices > 1) {
      const long long vectors = static_cast<long long>(M) * (K / 8);
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cfg.gridDim = dim3(static_cast<unsigned>((vectors + 127) / 128), 1, 1);
      cfg.blockDim = dim3(128, 1, 1);
      cfg.stream = s;
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaLaunchKernelEx(&cfg, glu_join_kernel, static_cast<const float*>(partial), slices,
                             static_cast<long long>(slice_size), static_cast<uint16_t*>(dX), ld.dx, K,
                             vectors) != cudaSuccess) {
        cudaGetLastError();
        st = GEMM_ERR_LAUNCH;
      } else {
        count_launch();
      }
    }
  }
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

}  // extern "C"
