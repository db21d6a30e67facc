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
//   dWg/dWu: A = dg or du, B = X, summed over the rows of X; one launch covers both.
// The gradient's products need operands along their other dimension (W by columns, dg and X by
// columns). The MMA takes them as they lie in memory: TMA boxes of 64 columns x 128 rows put the
// non-summed dimension innermost and the descriptors say so ("MN-major"), so nothing is transposed.
//
// A last wave of tiles at most half full runs as halves of its tiles (N = 128 MMAs).
// A stage holds 128 (BF16) or 256 (E4M3) of the summed dimension, 8 MMAs per barrier wait, 3 stages.
// Warp roles: 0 loads A, 2 loads B, 1 allocates TMEM and issues the MMAs (leader CTA), 4..7 epilogue,
// one TMEM lane quadrant each; stores go through swizzled staging tiles and TMA.
//
// Bound by the tensor cores for many rows and by the bytes of Wg and Wu for few.
//
// For the gradient g and u are kept in FP32 (8 bytes per element and a tenth of the block's time at
// most): kept in BF16 they would add a rounding to dg and du next to the one their MMA operand needs.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "glu_act.cuh"
#include "host_common.h"

namespace dtcp {

enum GluMode { kGluForward = 0, kGluForwardE4m3 = 1, kGluDx = 2, kGluDw = 3 };

struct GluParams {
  int rows, cols;        // of one output (dW: of dWg)
  int num_m_blocks, num_n_blocks, num_tiles, k_iters;
  int split_tiles, num_items;  // trailing tiles cut into halves of their columns; work items = tiles + split_tiles
  int depth;             // the summed dimension (dX: of one half)
  int half_blocks;       // dW: M-blocks of dWg; the ones after them are dWu's
  int half_iters;        // dX: stages of the first half
  int group_m;
  int act, save;
  const float* x_scale;  // E4M3: scales of X's rows, Wg's and Wu's
  const float* g_scale;
  const float* u_scale;
  unsigned* status;
  unsigned long long wait_limit_ns;
};

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
  static constexpr int WARP_A = 0, WARP_MMA = 1, WARP_B = 2, EPI_WARP0 = 4, EPI_WARPS = 4;
  static constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int EPI_BUFS = 2, EPI_BUF_BYTES = 32 * 128;  // 32 rows of 128 bytes
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = STAGES * OPERAND_BYTES;
  static constexpr int OFF_EPI = OFF_B + STAGES * OPERAND_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + EPI_WARPS * EPI_BUFS * EPI_BUF_BYTES;
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;  // slack to align the base to 1024 bytes
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(OFF_EPI % 1024 == 0, "1024-byte alignment");
};

namespace {

// Instruction descriptor (see idesc_bf16): BF16 operands, bits 15 / 16: A / B has its M / N dimension innermost.
__host__ __device__ constexpr uint32_t idesc_glu(int m, int n, bool a_mn, bool b_mn) {
  return idesc_bf16(m, n) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}
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

// Descriptor of an operand with its M (or N) dimension innermost, as a TMA box of 64 columns x 128
// rows with 128-byte swizzle leaves it: 8 rows of the summed dimension are 1024 bytes (the stride
// offset), the next 64 columns are the next box (the leading offset).
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t smem_addr) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>(GluLayout::ATOM_BYTES >> 4) << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// ---------------------------------------------------------------- producers (warps 0, 2)

template <int MODE>
__device__ __forceinline__ void glu_producer(const GluParams& p, const CUtensorMap* m0, const CUtensorMap* m1,
                                             uint32_t base, uint32_t rank, bool load_a, int cluster_idx,
                                             int num_clusters, const WaitCtx& wctx) {
  using L = GluLayout;
  constexpr int STAGE_K = MODE == kGluForwardE4m3 ? 256 : 128;
  constexpr bool A_MN = MODE == kGluDw, B_MN = MODE == kGluDx || MODE == kGluDw;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t dst0 = base + (load_a ? L::OFF_A : L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  int it = 0;
  for (int i = cluster_idx; i < p.num_items && ok; i += num_clusters, ++it) {
    const WorkItem w = work_item(i, p.num_tiles, p.split_tiles);
    const TileCoord tc = tile_coord(w.tile, p.num_m_blocks, p.num_n_blocks, p.group_m);
    const int half = w.half > 0 ? 1 : 0;
    const int b_boxes = w.half >= 0 ? 1 : 2;  // of 64 rows (K-major: per atom) or 64 columns (MN-major)
    const uint32_t stage_bytes = L::OPERAND_BYTES + L::OPERAND_BYTES / 2 * b_boxes;
    const bool down = (it & 1) != 0;  // start on the blocks the last wave of tiles read last
    const CUtensorMap* map = m0;
    int first;  // the operand's first row (K-major) or column (MN-major)
    if (load_a) {
      int mb = tc.m_blk;
      if (MODE == kGluDw && mb >= p.half_blocks) {
        mb -= p.half_blocks;
        map = m1;
      }
      first = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M;
    } else if (MODE == kGluForward || MODE == kGluForwardE4m3) {
      if (rank == 1) map = m1;
      first = tc.n_blk * L::FEATURES + half * (L::FEATURES / 2);
    } else {
      first = tc.n_blk * L::BLOCK_N + half * (L::BLOCK_N / 2) + static_cast<int>(rank) * 64 * b_boxes;
    }
    for (int kb = 0; kb < p.k_iters; ++kb) {
      if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
        ok = false;
        break;
      }
      int k = down ? p.k_iters - 1 - kb : kb;
      if (MODE == kGluDx) {
        map = k >= p.half_iters ? m1 : m0;
        if (k >= p.half_iters) k -= p.half_iters;
      }
      const uint32_t full = bar_full + 8 * stage;
      if (load_a && rank == 0) mbar_arrive_expect_tx(full, 2u * stage_bytes);
      const uint32_t bar = mapa_shared(full, 0);
      const uint32_t dst = dst0 + stage * L::OPERAND_BYTES;
      if (load_a ? A_MN : B_MN) {
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
  constexpr bool A_MN = MODE == kGluDw, B_MN = MODE == kGluDx || MODE == kGluDw, E4M3 = MODE == kGluForwardE4m3;
  constexpr int STAGE_K = E4M3 ? 256 : 128, MMA_K = E4M3 ? 32 : 16;
  constexpr uint32_t IDESC_FULL = E4M3 ? idesc_e4m3(256, L::BLOCK_N) : idesc_glu(256, L::BLOCK_N, A_MN, B_MN);
  constexpr uint32_t IDESC_HALF = E4M3 ? idesc_e4m3(256, L::BLOCK_N / 2) : idesc_glu(256, L::BLOCK_N / 2, A_MN, B_MN);
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  const uint64_t a0 = A_MN ? umma_desc_mn(base + L::OFF_A) : umma_desc_sw128(base + L::OFF_A);
  const uint64_t b0 = B_MN ? umma_desc_mn(base + L::OFF_B) : umma_desc_sw128(base + L::OFF_B);
  // MMA kk of a stage: K-major operands advance 32 bytes inside the swizzle row, four per atom;
  // MN-major ones by 16 rows of 128 bytes.
  auto step = [&](bool mn, int kk) -> uint32_t {
    return mn ? static_cast<uint32_t>(kk) * 2048u : static_cast<uint32_t>((kk / 4) * L::ATOM_BYTES + (kk % 4) * 32);
  };
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  int it = 0;
  for (int i = cluster_idx; i < p.num_items && ok; i += num_clusters, ++it) {
    const uint32_t idesc = work_item(i, p.num_tiles, p.split_tiles).half >= 0 ? IDESC_HALF : IDESC_FULL;
    const bool down = (it & 1) != 0;
    const uint32_t slot = static_cast<uint32_t>(it) & 1u;
    if (!wait_phase_inline(bar_tempty + 8 * slot, ((static_cast<uint32_t>(it) >> 1) & 1u) ^ 1u, wctx,
                           status_code(kRoleMma, 0x100 + slot))) {
      ok = false;
      break;
    }
    const uint32_t d = tmem_base + slot * L::ACC_COLS;
    for (int kb = 0; kb < p.k_iters; ++kb) {
      if (!wait_phase_inline(bar_full + 8 * stage, phase, wctx, status_code(kRoleMma, stage))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      int k = down ? p.k_iters - 1 - kb : kb;
      if (MODE == kGluDx && k >= p.half_iters) k -= p.half_iters;
      const uint64_t a = umma_desc_advance(a0, stage * L::OPERAND_BYTES);
      const uint64_t b = umma_desc_advance(b0, stage * L::OPERAND_BYTES);
      const int left = p.depth - k * STAGE_K;  // a ragged last stage: only the MMAs that hold any of it
      const int steps = left >= STAGE_K ? L::KSTEPS : (left + MMA_K - 1) / MMA_K;
      auto one = [&](int kk) {
        const uint64_t ad = umma_desc_advance(a, step(A_MN, kk)), bd = umma_desc_advance(b, step(B_MN, kk));
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

// ---------------------------------------------------------------- epilogue (warps 4..7)

// The warp's two staging buffers in turn; each is free once the store before last has read it.
struct GluStaging {
  uint32_t base, next;
  __device__ __forceinline__ uint32_t take(uint32_t lane) {
    const uint32_t buf = base + next * GluLayout::EPI_BUF_BYTES;
    next ^= 1u;
    if (lane == 0) bulk_wait_group_read<1>();
    __syncwarp();
    return buf;
  }
  __device__ __forceinline__ void store(uint32_t lane, const CUtensorMap* map, uint32_t buf, int col, int row) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(map, buf, col, row);
      bulk_commit_group();
    }
  }
};

// 32 columns of this lane's row as BF16 (64-byte rows, 64-byte swizzle).
__device__ __forceinline__ void glu_store_bf16(GluStaging& st, uint32_t lane, const CUtensorMap* map, const float (&v)[32],
                                               int col, int row) {
  const uint32_t buf = st.take(lane);
  const uint32_t addr = buf + lane * 64u, sw = (lane >> 1) & 3u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t w[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
      w[t] = pack_bf16x2_rn(__float_as_uint(v[8 * j + 2 * t]), __float_as_uint(v[8 * j + 2 * t + 1]));
    st_shared_v4(addr + ((static_cast<uint32_t>(j) ^ sw) << 4), w[0], w[1], w[2], w[3]);
  }
  st.store(lane, map, buf, col, row);
}

// 32 columns of this lane's row as FP32 (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ void glu_store_f32(GluStaging& st, uint32_t lane, const CUtensorMap* map,
                                              const uint32_t (&v)[32], int col, int row) {
  const uint32_t buf = st.take(lane);
  const uint32_t addr = buf + lane * 128u, sw = lane & 7u;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    st_shared_v4(addr + ((static_cast<uint32_t>(j) ^ sw) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  st.store(lane, map, buf, col, row);
}

template <int MODE>
__device__ __forceinline__ void glu_epilogue(const GluParams& p, const CUtensorMap* c0, const CUtensorMap* c1,
                                             const CUtensorMap* pre_g, const CUtensorMap* pre_u, uint32_t base,
                                             uint32_t tmem_base, uint32_t warp, uint32_t lane, uint32_t rank,
                                             int cluster_idx, int num_clusters, const WaitCtx& wctx) {
  using L = GluLayout;
  constexpr bool FORWARD = MODE == kGluForward || MODE == kGluForwardE4m3;
  const uint32_t bar_tfull = base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 16;
  const uint32_t q = warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
  const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
  GluStaging st{base + L::OFF_EPI + q * L::EPI_BUFS * L::EPI_BUF_BYTES, 0u};
  int it = 0;
  for (int i = cluster_idx; i < p.num_items; i += num_clusters, ++it) {
    const WorkItem w = work_item(i, p.num_tiles, p.split_tiles);
    const TileCoord tc = tile_coord(w.tile, p.num_m_blocks, p.num_n_blocks, p.group_m);
    const int columns = w.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;  // of the item's accumulator
    const int col0 = tc.n_blk * (FORWARD ? L::FEATURES : L::BLOCK_N) + (w.half > 0 ? columns / (FORWARD ? 2 : 1) : 0);
    const uint32_t slot = static_cast<uint32_t>(it) & 1u;
    // E4M3: this lane's row scale and its features' scales, while the MMAs run
    float x_scale = 1.0f, w_scale[2][L::FEATURES / 32];
    if constexpr (MODE == kGluForwardE4m3) {
      const int row = tc.m_blk * L::TILE_M + static_cast<int>(rank) * L::CTA_M + static_cast<int>(q * 32 + lane);
      if (row < p.rows) x_scale = p.x_scale[row];
#pragma unroll
      for (int c = 0; c < L::FEATURES / 32; ++c) {
        const int f = col0 + c * 32 + static_cast<int>(lane);
        w_scale[0][c] = f < p.cols ? p.g_scale[f] : 0.0f;
        w_scale[1][c] = f < p.cols ? p.u_scale[f] : 0.0f;
      }
    }
    if (!wait_phase_warp(bar_tfull + 8 * slot, (static_cast<uint32_t>(it) >> 1) & 1u, wctx,
                         status_code(kRoleEpilogue, slot)))
      break;
    tc_fence_after_sync();
    int mb = tc.m_blk;
    const CUtensorMap* out = c0;
    if (MODE == kGluDw && mb >= p.half_blocks) {
      mb -= p.half_blocks;
      out = c1;
    }
    const int row0 = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M + static_cast<int>(q) * 32;
    const uint32_t taddr = tmem_base + ((q * 32u) << 16) + slot * L::ACC_COLS;
    if (row0 < p.rows) {
      if constexpr (FORWARD) {
        const float xs = x_scale;
#pragma unroll MODE == kGluForwardE4m3 ? 4 : 1
        for (int c = 0; c < L::FEATURES; c += 32) {
          const int col = col0 + c;
          if (c >= columns / 2 || col >= p.cols) break;
          float gs = 0.0f, us = 0.0f;  // E4M3: the scales of feature col + lane
          if constexpr (MODE == kGluForwardE4m3) {
            gs = w_scale[0][c / 32];
            us = w_scale[1][c / 32];
          }
          uint32_t g[32], u[32];
          tmem_ld_32x32b_x32(taddr + c, g);
          tmem_ld_32x32b_x32(taddr + columns / 2 + c, u);
          tmem_ld_wait();
          float h[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float gv = __uint_as_float(g[j]), uv = __uint_as_float(u[j]);
            if constexpr (MODE == kGluForwardE4m3) {
              gv *= xs * __shfl_sync(0xffffffffu, gs, j);
              uv *= xs * __shfl_sync(0xffffffffu, us, j);
            }
            h[j] = glu_act(gv, p.act) * uv;
          }
          glu_store_bf16(st, lane, out, h, col, row0);
          if (p.save) {
            glu_store_f32(st, lane, pre_g, g, col, row0);
            glu_store_f32(st, lane, pre_u, u, col, row0);
          }
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < columns; c += 32) {
          const int col = col0 + c;
          if (col >= p.cols) break;
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c, v);
          tmem_ld_wait();
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]);
          glu_store_bf16(st, lane, out, f, col, row0);
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
    glu_kernel(const __grid_constant__ CUtensorMap a0, const __grid_constant__ CUtensorMap a1,
               const __grid_constant__ CUtensorMap b0, const __grid_constant__ CUtensorMap b1,
               const __grid_constant__ CUtensorMap c0, const __grid_constant__ CUtensorMap c1,
               const __grid_constant__ CUtensorMap pre_g, const __grid_constant__ CUtensorMap pre_u, const GluParams p) {
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
      if (warp == L::WARP_A) glu_producer<MODE>(p, &a0, &a1, base, rank, true, cluster_idx, num_clusters, wctx);
      else if (warp == L::WARP_B) glu_producer<MODE>(p, &b0, &b1, base, rank, false, cluster_idx, num_clusters, wctx);
      else if (warp == L::WARP_MMA && rank == 0) glu_mma<MODE>(p, base, tmem_base, cluster_idx, num_clusters, wctx);
    }
    __syncwarp();
  } else {
    glu_epilogue<MODE>(p, &c0, &c1, &pre_g, &pre_u, base, tmem_base, warp, lane, rank, cluster_idx, num_clusters, wctx);
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
    const float4 ga = gp[0], gb = gp[1], ua = up[0], ub = up[1];
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

// ---------------------------------------------------------------- host side

struct GluMaps {
  CUtensorMap a0, a1, b0, b1, c0, c1, pre_g, pre_u;
};

int glu_max_clusters(int device) {
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (cache[device] > 0) return cache[device];
  for (auto k : {glu_kernel<kGluForward>, glu_kernel<kGluForwardE4m3>, glu_kernel<kGluDx>, glu_kernel<kGluDw>})
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

// B's boxes are half its rows, so that a half tile's load is one box.
int map_kb(CUtensorMap* m, const void* p, int depth, int rows) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, depth, rows, uint64_t(depth) * 2, 64, 64,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}
// A BF16 operand with the summed dimension along its rows (K-major) or along its columns (MN-major).
int map_k(CUtensorMap* m, const void* p, int depth, int rows, long long ld) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, depth, rows, uint64_t(ld) * 2, 64, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}
int map_mn(CUtensorMap* m, const void* p, int cols, int depth, long long ld) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, depth, uint64_t(ld) * 2, 64, 128,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}
int map_out(CUtensorMap* m, const void* p, int cols, int rows, long long ld) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, rows, uint64_t(ld) * 2, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_64B);
}

// The tiles of a rows x cols output (virtual sizes in units of the 256 x 256 tile's operands) on the co-resident pairs.
template <int MODE>
int glu_launch(GluMaps& m, GluParams& p, int virtual_rows, int virtual_cols, int virtual_depth, double bytes, int device,
               const DeviceInfo* info, cudaStream_t stream) {
  using L = GluLayout;
  const long long tiles = static_cast<long long>(p.num_m_blocks) * p.num_n_blocks;
  if (tiles > 0x3FFFFFFFLL) return GEMM_ERR_UNSUPPORTED_SHAPE;
  p.num_tiles = static_cast<int>(tiles);
  p.status = device_status_word(device);
  p.wait_limit_ns = RunOptions().wait_limit_ns;
  if (p.status == nullptr) return GEMM_ERR_NO_DEVICE;
  const int max_clusters = glu_max_clusters(device);
  if (max_clusters <= 0) return GEMM_ERR_LAUNCH;
  p.split_tiles = tail_split_tiles(p.num_tiles, max_clusters);
  p.num_items = p.num_tiles + p.split_tiles;
  const int clusters = std::min(p.num_items, max_clusters);
  p.group_m = choose_group_m(virtual_rows, virtual_cols, virtual_depth, L::TILE_M, L::BLOCK_N, bytes, 0.0, clusters,
                             info->l2_bytes);
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
  if (cudaLaunchKernelEx(&cfg, glu_kernel<MODE>, m.a0, m.a1, m.b0, m.b1, m.c0, m.c1, m.pre_g, m.pre_u, p) !=
      cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
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
  if (M <= kGluFewRows) {
    GluFewParams f = {X, Wg, Wu, static_cast<uint16_t*>(H), preact, nullptr, nullptr, nullptr, ld.x, ld.h, M, N, K, act};
    return run_glu_few(f, false, s);
  }
  GluMaps m;
  GluParams p = {};
  int st = map_k(&m.a0, X, K, M, ld.x);
  if (st == GEMM_OK) st = map_kb(&m.b0, Wg, K, N);
  if (st == GEMM_OK) st = map_kb(&m.b1, Wu, K, N);
  if (st == GEMM_OK) st = map_out(&m.c0, H, N, M, ld.h);
  if (st != GEMM_OK) return st;
  m.a1 = m.a0;
  m.c1 = m.pre_g = m.pre_u = m.c0;
  if (preact != nullptr) {
    st = encode_tmap_2d(&m.pre_g, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, preact, N, M, uint64_t(N) * 8, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == GEMM_OK)
      st = encode_tmap_2d(&m.pre_u, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, preact + N, N, M, uint64_t(N) * 8, 32, 32,
                          CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != GEMM_OK) return st;
  }
  p.rows = M;
  p.cols = N;
  p.depth = K;
  p.num_m_blocks = ceil_div(M, L::TILE_M);
  p.num_n_blocks = ceil_div(N, L::FEATURES);
  p.k_iters = ceil_div(K, 128);
  p.act = act;
  p.save = preact != nullptr ? 1 : 0;
  const int virtual_cols = static_cast<int>(std::min<long long>(2LL * N, 0x7FFFFFFF));
  return glu_launch<kGluForward>(m, p, M, virtual_cols, K, 2.0, device, info, s);
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
  if (!aligned16(H) || (K > 0 && (!aligned16(X) || !aligned16(Wg) || !aligned16(Wu) ||
                                  (reinterpret_cast<uintptr_t>(x_scale) & 3u) || (reinterpret_cast<uintptr_t>(wg_scale) & 3u) ||
                                  (reinterpret_cast<uintptr_t>(wu_scale) & 3u))))
    return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (K == 0) return zero_rows(H, size_t(N) * 2, ld.h * 2, M, s);
  if (M <= kGluFewRowsE4m3) {
    GluFewParams f = {X, Wg, Wu, static_cast<uint16_t*>(H), nullptr, x_scale, wg_scale, wu_scale, ld.x, ld.h, M, N, K, act};
    return run_glu_few(f, true, s);
  }
  GluMaps m;
  GluParams p = {};
  auto map8 = [&](CUtensorMap* t, const void* q, int rows, long long stride, int box_rows) {
    return encode_tmap_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, rows, stride, 128, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  int st = map8(&m.a0, X, M, ld.x, 128);
  if (st == GEMM_OK) st = map8(&m.b0, Wg, N, K, 64);
  if (st == GEMM_OK) st = map8(&m.b1, Wu, N, K, 64);
  if (st == GEMM_OK) st = map_out(&m.c0, H, N, M, ld.h);
  if (st != GEMM_OK) return st;
  m.a1 = m.a0;
  m.c1 = m.pre_g = m.pre_u = m.c0;
  p.rows = M;
  p.cols = N;
  p.depth = K;
  p.num_m_blocks = ceil_div(M, L::TILE_M);
  p.num_n_blocks = ceil_div(N, L::FEATURES);
  p.k_iters = ceil_div(K, 256);
  p.act = act;
  p.x_scale = x_scale;
  p.g_scale = wg_scale;
  p.u_scale = wu_scale;
  const int virtual_cols = static_cast<int>(std::min<long long>(2LL * N, 0x7FFFFFFF));
  return glu_launch<kGluForwardE4m3>(m, p, M, virtual_cols, K, 1.0, device, info, s);
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
  cudaMemPool_t pool = workspace_pool(device);
  void* ws = nullptr;
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, size_t(M) * N * 4, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  uint16_t* dgu = static_cast<uint16_t*>(ws);
  int st;
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
  if (st == GEMM_OK && dX != nullptr) {
    GluMaps m;
    GluParams p = {};
    st = map_k(&m.a0, dgu, N, M, 2LL * N);
    if (st == GEMM_OK) st = map_k(&m.a1, dgu + N, N, M, 2LL * N);
    if (st == GEMM_OK) st = map_mn(&m.b0, Wg, K, N, K);
    if (st == GEMM_OK) st = map_mn(&m.b1, Wu, K, N, K);
    if (st == GEMM_OK) st = map_out(&m.c0, dX, K, M, ld.dx);
    if (st == GEMM_OK) {
      m.c1 = m.pre_g = m.pre_u = m.c0;
      p.rows = M;
      p.cols = K;
      p.depth = N;
      p.num_m_blocks = ceil_div(M, L::TILE_M);
      p.num_n_blocks = ceil_div(K, L::BLOCK_N);
      p.half_iters = ceil_div(N, 128);
      p.k_iters = 2 * p.half_iters;
      st = glu_launch<kGluDx>(m, p, M, K, 2 * N, 2.0, device, info, s);
    }
  }
  if (st == GEMM_OK && dWg != nullptr) {
    GluMaps m;
    GluParams p = {};
    st = map_mn(&m.a0, dgu, N, M, 2LL * N);
    if (st == GEMM_OK) st = map_mn(&m.a1, dgu + N, N, M, 2LL * N);
    if (st == GEMM_OK) st = map_mn(&m.b0, X, K, M, ld.x);
    if (st == GEMM_OK) st = map_out(&m.c0, dWg, K, N, K);
    if (st == GEMM_OK) st = map_out(&m.c1, dWu, K, N, K);
    if (st == GEMM_OK) {
      m.b1 = m.b0;
      m.pre_g = m.pre_u = m.c0;
      p.rows = N;
      p.cols = K;
      p.depth = M;
      p.half_blocks = ceil_div(N, L::TILE_M);
      p.num_m_blocks = 2 * p.half_blocks;
      p.num_n_blocks = ceil_div(K, L::BLOCK_N);
      p.k_iters = ceil_div(M, 128);
      st = glu_launch<kGluDw>(m, p, 2 * N, K, M, 2.0, device, info, s);
    }
  }
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

}  // extern "C"
