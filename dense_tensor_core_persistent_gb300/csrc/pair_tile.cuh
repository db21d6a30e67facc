// pair_tile.cuh -- the persistent, warp-specialised tensor-core pipelines that the operators around the products share: a
// 256 x 256 and a 512 x 256 output tile per CTA pair, their work items, tensor maps, operand descriptors, loads and MMAs.
// An operator brings the epilogue and launches (glu.cu, glu_wide.cu, pair_gradient.cu, cross_entropy.cu).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "host_common.h"

namespace dtcp {

// What the operands of a launch are.
enum PairMode {
  kPairGated = 0,      // A: rows of X; B: 128 rows of Wg over the same 128 of Wu
  kPairGatedE4m3 = 1,  // the same in E4M3 (256 x 256 tile only)
  kPairGradient = 2,   // main: A = rows of G (K-major), B = W by columns; second: A = G, B = X, both by columns
  kPairRows = 3        // A: rows of X; B: 256 rows of W; the depth in parts of kPairSumStages stages with an accumulator each,
                       // which the epilogue adds in FP32 (256 x 256 tile only)
};

// A tensor-core step cuts what lies below its FP32 accumulator's last place, so a long sum in one accumulator shrinks
// towards zero by some 2^-25 a step. Logits, which stay in FP32, are summed in parts of 512. Measured on GB300, cross entropy
// of 1500 x 50001 x 2056 and 4096 x 131072 x 4096 (error of lse against 64 bits): one part 1% faster (1.2e-6), parts of 512
// (2.5e-7), parts of 256 2 to 3% slower (1.2e-7).
constexpr int kPairSumStages = 4;

// The tiles of one product: rows x cols of output, the summed dimension `depth` (dX: of one half) in `k_iters` stages.
struct PairProduct {
  int rows, cols, depth, k_iters;
  int num_m_blocks, num_n_blocks, num_tiles, group_m;
  int split_tiles, num_items;  // trailing tiles cut into halves of their columns; work items = tiles + split_tiles
  int slices;                  // parts of the summed dimension, each an item of its own (then no halves)
  int slice_rows;              // rows from one slice's partial sums to the next one's
};

struct PairParams {
  PairProduct main;    // forward: the output; gradient: dX
  PairProduct second;  // gradient: dW (rows and blocks of all its parts)
  int parts;           // gradient: 2 if G is [G0 | G1] and W is [W0 ; W1] in two tensors (dX sums over both), else 1
  int ahead;           // gradient: items of `second` that each cluster without a tile in dX's last wave takes meanwhile
  unsigned* status;
  unsigned long long wait_limit_ns;
};

// One work item.
struct PairItem {
  int m_blk, n_blk, half;
  bool second;
  int slice, k0, k1;  // its stages
};

// Item `it` of a cluster; false past its last one.
__device__ __forceinline__ bool pair_item(const PairParams& p, int cluster, int clusters, int it, PairItem& item) {
  const PairProduct* q = &p.main;
  int i = cluster + it * clusters;
  item.second = i >= p.main.num_items;
  if (item.second) {
    q = &p.second;
    const int in_last = p.main.num_items % clusters;  // clusters with a tile in the last wave of the first product
    const int before = p.main.num_items / clusters + (cluster < in_last ? 1 : 0);
    int s = it - before;
    const int extra = in_last > 0 && cluster >= in_last ? p.ahead : 0;
    const int taken = in_last > 0 ? p.ahead * (clusters - in_last) : 0;
    i = s < extra ? s * (clusters - in_last) + cluster - in_last : taken + (s - extra) * clusters + cluster;
    if (i >= p.second.num_items) return false;
  }
  item.slice = 0;
  if (q->slices > 1) {
    item.slice = i / q->num_tiles;
    i -= item.slice * q->num_tiles;
  }
  item.k0 = item.slice * q->k_iters / q->slices;
  item.k1 = (item.slice + 1) * q->k_iters / q->slices;
  const WorkItem w = work_item(i, q->num_tiles, q->split_tiles);
  const TileCoord tc = tile_coord(w.tile, q->num_m_blocks, q->num_n_blocks, q->group_m);
  item.m_blk = tc.m_blk;
  item.n_blk = tc.n_blk;
  item.half = w.half;
  return true;
}

struct PairMaps {
  CUtensorMap a0, a1;      // forward: X (both); gradient: G's parts
  CUtensorMap b0, b1, b2;  // gated: Wg, Wu; rows: W (b0); gradient: W's parts, X
  CUtensorMap c0, c1, c2;  // gated: H, g, u; gradient: dX (or its partial sums), dW's parts
};

// Instruction descriptor (see idesc_bf16): BF16 operands, bits 15 / 16: A / B has its M / N dimension innermost.
__host__ __device__ constexpr uint32_t idesc_mn(int m, int n, bool a_mn, bool b_mn) {
  return idesc_bf16(m, n) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}
// Descriptor of an operand with its M (or N) dimension innermost, as TMA boxes of 64 columns with 128-byte swizzle
// leave it: 8 rows of the summed dimension are 1024 bytes (the stride offset), the next 64 columns are the next box,
// `box_bytes` on (the leading offset).
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t smem_addr, uint32_t box_bytes) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(box_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// 2-D tile store of data that is not read again soon: it leaves L2 first, before the operands that are read again.
__device__ __forceinline__ void tma_store_2d_streaming(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y) {
  asm volatile(
      "{\n\t.reg .b64 policy;\n\t"
      "createpolicy.fractional.L2::evict_first.b64 policy, 1.0;\n\t"
      "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3}], [%1], policy;\n\t}"
      ::"l"(m), "r"(src), "r"(x), "r"(y)
      : "memory");
}

// 2-D tile of FP32 added to what is in memory (each element once: the order of a launch's adds does not matter).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* m, uint32_t src, int32_t x, int32_t y) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m),
               "r"(src), "r"(x), "r"(y)
               : "memory");
}

// How a tile reaches memory: a plain store, one that leaves L2 first, or added to what is there (FP32).
enum PairStore { kPairPlain = 0, kPairStreaming = 1, kPairAdd = 2 };

// An epilogue warp's staging bytes: two BF16 tiles of 32 x 32 in turn, or (`whole`) one tile, FP32 or BF16, at a time.
constexpr int kPairStagingBytes = 32 * 128;
struct PairStaging {
  uint32_t base, next;
  bool whole;
  __device__ __forceinline__ uint32_t take(uint32_t lane) {
    uint32_t buf = base;
    if (whole) {
      if (lane == 0) bulk_wait_group_read<0>();
    } else {
      buf += next * (kPairStagingBytes / 2);
      next ^= 1u;
      if (lane == 0) bulk_wait_group_read<1>();
    }
    __syncwarp();
    return buf;
  }
  __device__ __forceinline__ void store(uint32_t lane, const CUtensorMap* map, uint32_t buf, int col, int row,
                                        PairStore how) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (how == kPairStreaming) tma_store_2d_streaming(map, buf, col, row);
      else if (how == kPairAdd) tma_add_2d(map, buf, col, row);
      else tma_store_2d(map, buf, col, row);
      bulk_commit_group();
    }
  }
};

// 32 columns of this lane's row as BF16 (64-byte rows, 64-byte swizzle) or FP32 (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ void pair_store(PairStaging& st, uint32_t lane, const CUtensorMap* map, const uint32_t (&v)[32],
                                          int col, int row, bool f32, PairStore how = kPairPlain) {
  const uint32_t buf = st.take(lane);
  if (f32) {
    const uint32_t addr = buf + lane * 128u, sw = lane & 7u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      st_shared_v4(addr + ((static_cast<uint32_t>(j) ^ sw) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    const uint32_t addr = buf + lane * 64u, sw = (lane >> 1) & 3u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      st_shared_v4(addr + ((static_cast<uint32_t>(j) ^ sw) << 4), pack_bf16x2_rn(v[8 * j], v[8 * j + 1]),
                   pack_bf16x2_rn(v[8 * j + 2], v[8 * j + 3]), pack_bf16x2_rn(v[8 * j + 4], v[8 * j + 5]),
                   pack_bf16x2_rn(v[8 * j + 6], v[8 * j + 7]));
  }
  st.store(lane, map, buf, col, row, how);
}

// ---------------------------------------------------------------- the 256 x 256 tile

// Registers per thread of a launch of 384 threads (65536 / 384 -> 168), and after setmaxnreg.
constexpr int kPairRegsLaunch = 168, kPairRegsLow = 56, kPairRegsEpilogue = 216;

struct PairLayout {
  static constexpr int CG = 2;
  static constexpr int CTA_M = 128, TILE_M = 256;
  static constexpr int BLOCK_N = 256, B_ROWS = 128;  // B rows each CTA loads
  static constexpr int FEATURES = 128;               // gated: features of a tile
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
  static constexpr int OFF_BAR = OFF_EPI + EPI_WARPS * kPairStagingBytes;
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;  // slack to align the base to 1024 bytes
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
  static_assert(OFF_EPI % 1024 == 0, "1024-byte alignment");
};

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

// Producers (warps 0, 2).
template <int MODE>
__device__ __forceinline__ void pair_producer(const PairParams& p, const PairMaps& maps, uint32_t base, uint32_t rank,
                                             bool load_a, int cluster_idx, int num_clusters, const WaitCtx& wctx) {
  using L = PairLayout;
  constexpr bool GRADIENT = MODE == kPairGradient;
  constexpr int STAGE_K = MODE == kPairGatedE4m3 ? 256 : 128;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t dst0 = base + (load_a ? L::OFF_A : L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  PairItem item;
  for (int it = 0; ok && pair_item(p, cluster_idx, num_clusters, it, item); ++it) {
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
        const int part_blocks = p.second.num_m_blocks / p.parts;
        if (mb >= part_blocks) {
          mb -= part_blocks;
          m0 = m1;
        }
      }
      first = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M;
      mn = GRADIENT && item.second;
    } else if (MODE == kPairRows) {
      m0 = m1 = &maps.b0;
      first = item.n_blk * L::BLOCK_N + half * (L::BLOCK_N / 2) + static_cast<int>(rank) * 64 * b_boxes;
      mn = false;
    } else if (!GRADIENT) {
      m0 = m1 = rank == 1 ? &maps.b1 : &maps.b0;
      first = item.n_blk * L::FEATURES + half * (L::FEATURES / 2);
      mn = false;
    } else {
      m0 = item.second ? &maps.b2 : &maps.b0;
      m1 = &maps.b1;
      first = item.n_blk * L::BLOCK_N + half * (L::BLOCK_N / 2) + static_cast<int>(rank) * 64 * b_boxes;
      mn = true;
    }
    const int part_iters = GRADIENT && !item.second ? k_iters / p.parts : k_iters;
    for (int kb = 0; kb < item.k1 - item.k0; ++kb) {
      if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
        ok = false;
        break;
      }
      int k = down ? item.k1 - 1 - kb : item.k0 + kb;
      const CUtensorMap* map = m0;
      if (k >= part_iters) {
        k -= part_iters;
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

// MMA issuer (leader, warp 1).
template <int MODE>
__device__ __forceinline__ void pair_mma(const PairParams& p, uint32_t base, uint32_t tmem_base, int cluster_idx,
                                        int num_clusters, const WaitCtx& wctx) {
  using L = PairLayout;
  constexpr bool GRADIENT = MODE == kPairGradient, E4M3 = MODE == kPairGatedE4m3;
  constexpr int STAGE_K = E4M3 ? 256 : 128, MMA_K = E4M3 ? 32 : 16;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  const uint64_t a_k = umma_desc_sw128(base + L::OFF_A), a_mn = umma_desc_mn(base + L::OFF_A, L::ATOM_BYTES);
  const uint64_t b0 = GRADIENT ? umma_desc_mn(base + L::OFF_B, L::ATOM_BYTES) : umma_desc_sw128(base + L::OFF_B);
  constexpr bool SUMS = MODE == kPairRows;
  uint32_t stage = 0, phase = 0;
  int acc = 0;  // accumulators taken: one an item, or one for each part of its depth
  bool ok = true;
  PairItem item;
  for (int it = 0; ok && pair_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const bool dw = GRADIENT && item.second;
    const uint32_t n = item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;
    const uint32_t idesc = E4M3 ? idesc_e4m3(256, n) : idesc_mn(256, n, dw, GRADIENT);
    const bool down = (it & 1) != 0;
    const PairProduct& q = item.second ? p.second : p.main;
    const int part_iters = GRADIENT && !item.second ? q.k_iters / p.parts : q.k_iters;
    uint32_t slot = 0, d = 0;
    for (int kb = 0; kb < item.k1 - item.k0; ++kb) {
      const int in_part = SUMS ? kb % kPairSumStages : kb;
      if (in_part == 0) {
        slot = static_cast<uint32_t>(acc) & 1u;
        d = tmem_base + slot * L::ACC_COLS;
        if (!wait_phase_inline(bar_tempty + 8 * slot, ((static_cast<uint32_t>(acc) >> 1) & 1u) ^ 1u, wctx,
                               status_code(kRoleMma, 0x100 + slot))) {
          ok = false;
          break;
        }
        ++acc;
      }
      if (!wait_phase_inline(bar_full + 8 * stage, phase, wctx, status_code(kRoleMma, stage))) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      int k = down ? item.k1 - 1 - kb : item.k0 + kb;
      if (k >= part_iters) k -= part_iters;
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
        const uint64_t bd = umma_desc_advance(b, GRADIENT ? step_mn : step_k);
        if constexpr (E4M3) mma_e4m3_pair(d, ad, bd, idesc, (in_part | kk) != 0 ? 1u : 0u);
        else mma_f16<2>(d, ad, bd, idesc, (in_part | kk) != 0 ? 1u : 0u);
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
      if (SUMS && in_part + 1 == kPairSumStages && kb + 1 < item.k1 - item.k0)
        mma_commit_pair_multicast(bar_tfull + 8 * slot, 0x3);
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

// What an epilogue warp knows of its CTA.
struct PairCta {
  uint32_t base, tmem_base, warp, lane, rank;
  int cluster_idx, num_clusters;
  WaitCtx wctx;
};

// All roles meet here once their work is done; the MMA warp (which allocated TMEM) frees it.
__device__ __forceinline__ void pair_teardown(uint32_t warp, uint32_t tmem_base) {
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == PairLayout::WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem_base, PairLayout::TMEM_COLS);
  }
}

// A CTA of the launch: set-up, roles, teardown. Warps from EPI_WARP0 on run `epilogue`; where it adds parts in registers,
// the producer warpgroup gives up some of its own (as on the 512 x 256 tile).
template <int MODE, class Epilogue>
__device__ __forceinline__ void pair_cta(const PairMaps& maps, const PairParams& p, Epilogue epilogue) {
  using L = PairLayout;
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

  // One branch per role group, each running to the end of the kernel (the code after a change of register limit
  // belongs to that limit).
  if (warp < L::EPI_WARP0) {
    if constexpr (MODE == kPairRows) regs_decrease<kPairRegsLow>();
    if (lane == 0) {
      if (warp == L::WARP_A || warp == L::WARP_B)
        pair_producer<MODE>(p, maps, base, rank, warp == L::WARP_A, cluster_idx, num_clusters, wctx);
      else if (warp == L::WARP_MMA && rank == 0)
        pair_mma<MODE>(p, base, tmem_base, cluster_idx, num_clusters, wctx);
    }
    __syncwarp();
    pair_teardown(warp, tmem_base);
  } else {
    if constexpr (MODE == kPairRows) regs_increase<kPairRegsEpilogue>();
    epilogue(PairCta{base, tmem_base, warp, lane, rank, cluster_idx, num_clusters, wctx});
    pair_teardown(warp, tmem_base);
  }
}

// ---------------------------------------------------------------- the 512 x 256 tile

struct PairWideLayout {
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
  static constexpr int REGS_LAUNCH = kPairRegsLaunch, REGS_LOW = kPairRegsLow, REGS_EPI = kPairRegsEpilogue;
  static constexpr int EPI_BYTES = kPairStagingBytes;
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

// Producers (warps 0, 2).
template <int MODE>
__device__ __forceinline__ void pair_wide_producer(const PairParams& p, const PairMaps& maps, uint32_t base, uint32_t rank,
                                                  bool load_a, int cluster_idx, int num_clusters, const WaitCtx& wctx) {
  using L = PairWideLayout;
  constexpr bool GRADIENT = MODE == kPairGradient;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t dst0 = base + (load_a ? L::OFF_A : L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  PairItem item;
  for (int it = 0; ok && pair_item(p, cluster_idx, num_clusters, it, item); ++it) {
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
      if (GRADIENT && item.second && mb >= p.second.num_m_blocks / p.parts) {
        mb -= p.second.num_m_blocks / p.parts;
        m0 = m1;
      }
      first = mb * L::TILE_M + static_cast<int>(rank) * L::CTA_M;
      mn = GRADIENT && item.second;
    } else if (!GRADIENT) {
      m0 = m1 = rank == 1 ? &maps.b1 : &maps.b0;
      first = item.n_blk * L::FEATURES + half * (L::FEATURES / 2);
      mn = false;
    } else {
      m0 = item.second ? &maps.b2 : &maps.b0;
      m1 = &maps.b1;
      first = item.n_blk * L::BLOCK_N + half * (L::BLOCK_N / 2) + static_cast<int>(rank) * 64 * b_boxes;
      mn = true;
    }
    const int part_iters = GRADIENT && !item.second ? k_iters / p.parts : k_iters;
    const int boxes = load_a ? L::A_BOXES : b_boxes;
    const uint32_t stride = load_a ? L::A_BYTES : L::B_BYTES;
    for (int kb = 0; kb < k_iters; ++kb) {
      if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
        ok = false;
        break;
      }
      int k = down ? k_iters - 1 - kb : kb;
      const CUtensorMap* map = m0;
      if (k >= part_iters) {
        k -= part_iters;
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

// MMA issuer (leader, warp 1).
template <int MODE>
__device__ __forceinline__ void pair_wide_mma(const PairParams& p, uint32_t base, uint32_t tmem_base, int cluster_idx,
                                             int num_clusters, const WaitCtx& wctx) {
  using L = PairWideLayout;
  constexpr bool GRADIENT = MODE == kPairGradient;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 8 * L::WAVES;
  const uint32_t bar_drain = bar_tempty + 8 * L::WAVES;
  const uint64_t a_k = umma_desc_sw128(base + L::OFF_A), a_mn = umma_desc_mn(base + L::OFF_A, L::BOX_BYTES);
  const uint64_t b0 = GRADIENT ? umma_desc_mn(base + L::OFF_B, L::BOX_BYTES) : umma_desc_sw128(base + L::OFF_B);
  uint32_t stage = 0, phase = 0;
  bool ok = true;
  PairItem item;
  for (int it = 0; ok && pair_item(p, cluster_idx, num_clusters, it, item); ++it) {
    const bool dw = GRADIENT && item.second;
    const uint32_t idesc = idesc_mn(256, item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N, dw, GRADIENT);
    const bool down = (it & 1) != 0;
    const uint32_t free_parity = (static_cast<uint32_t>(it) & 1u) ^ 1u;
    const PairProduct& q = item.second ? p.second : p.main;
    const int part_iters = GRADIENT && !item.second ? q.k_iters / p.parts : q.k_iters;
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
      if (k >= part_iters) k -= part_iters;
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
                     umma_desc_advance(b, GRADIENT ? step_mn : step_k), idesc, (kb | kk) != 0 ? 1u : 0u);
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

// All roles meet here once their work is done; the MMA warp (which allocated TMEM) frees it.
__device__ __forceinline__ void pair_wide_teardown(uint32_t warp, uint32_t tmem_base) {
  tc_fence_before_sync();
  cluster_sync_all();
  if (warp == PairWideLayout::WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc<2>(tmem_base, PairWideLayout::TMEM_COLS);
  }
}

// A CTA of the launch, as pair_cta.
template <int MODE, class Epilogue>
__device__ __forceinline__ void pair_wide_cta(const PairMaps& maps, const PairParams& p, Epilogue epilogue) {
  using L = PairWideLayout;
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
        pair_wide_producer<MODE>(p, maps, base, rank, warp == L::WARP_A, cluster_idx, num_clusters, wctx);
      else if (warp == L::WARP_MMA && rank == 0)
        pair_wide_mma<MODE>(p, base, tmem_base, cluster_idx, num_clusters, wctx);
    }
    __syncwarp();
    pair_wide_teardown(warp, tmem_base);
  } else {
    regs_increase<L::REGS_EPI>();
    epilogue(PairCta{base, tmem_base, warp, lane, rank, cluster_idx, num_clusters, wctx});
    pair_wide_teardown(warp, tmem_base);
  }
}

// ---------------------------------------------------------------- host side (pair_gradient.cu)

// Prepares a launch's kernels on the current device and gives the pairs that it holds at once (they agree: the shared
// memory bounds them); 0 on an error. The caller keeps the answer.
int pair_max_clusters(const void* const* kernels, int count, bool wide);

// A BF16 operand in boxes of 64 elements of its rows (the summed dimension if it is K-major, else columns) x `box_rows`.
int pair_map_in(CUtensorMap* m, const void* p, int cols, int rows, long long ld, int box_rows);
// Outputs, as pair_store stages them.
int pair_map_out(CUtensorMap* m, const void* p, int cols, int rows, long long ld);
int pair_map_out_f32(CUtensorMap* m, const void* p, int cols, uint64_t rows, long long ld);

// The tiles of a product; `rows` and `cols` are those of one output, of which `outputs` lie one after the other along
// the rows; tile_rows, cols_a_tile: rows of a pair's tile and output columns of its 256-column accumulator.
int pair_plan_product(PairProduct* q, int rows, int cols, int depth, int stage, int parts, int outputs, int tile_rows,
                      int cols_a_tile);

// Whether BF16 products of the given tiles (512 rows each; std: 256 rows) run on the 512 x 256 tile.
bool pair_wide_rule(long long std_tiles, long long wide_tiles, int depth, int wave);

// Fills in what a launch on `wave` co-resident pairs needs (halves of tiles, who goes ahead, orders; `bytes` per
// element of the operands) and gives its pairs; a negative status on an error.
// even: see PairGradient.
int pair_schedule(PairParams* p, bool wide, double bytes, int wave, int device, const DeviceInfo* info, bool even = false);

// Launches `kernel` with the arguments of `args` on `clusters` pairs.
int pair_launch(const void* kernel, void** args, bool wide, int clusters, cudaStream_t stream);

// dX = sum over the parts of G W and dW = G^T X in one launch.
struct PairGradient {
  const void *g[2], *w[2], *x;  // parts of G (rows x features, stride ldg) and of W (features x K); X: rows x K
  long long ldg, ldx, lddx;
  void *dx, *dw[2];  // either may be null
  int rows, features[2], K, parts;  // features[0] >= features[1]
  int most_slices;   // of dX's sum (0: no limit)
  bool even;         // the parts of dX's sum by an even share of the launch, and shallow tiles of dW by their store
  bool keep_sums;    // dX stays in `sums` (FP32), to be joined later
  bool add;          // and is added to what is there
};
struct PairGradientPlan {
  bool wide;
  PairParams p;
  size_t sums;  // floats of partial sums that dX needs (0: none)
};
// Whether it runs on the 512 x 256 tile, on `wave` co-resident pairs (only sizes and null pointers are looked at).
bool pair_gradient_is_wide(const PairGradient& q, int wave);
int pair_gradient_plan(const PairGradient& q, int device, PairGradientPlan* plan);
int pair_gradient_launch(const PairGradient& q, PairGradientPlan* plan, float* sums, int device, const DeviceInfo* info,
                         cudaStream_t stream);
// dX = bf16_rne(the slices' partial sums, added in their order). halves: the launch had 2 * rows rows, of which r and
// r + rows belong together.
int pair_gradient_join(const float* sums, int slices, void* dx, long long lddx, int rows, int K, cudaStream_t stream,
                       bool halves = false);

}  // namespace dtcp
