// glu_common.cuh -- what the gated feed-forward block's tensor-core kernels share: the products and their work items,
// tensor maps, and descriptors for operands with their M or N dimension innermost.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "host_common.h"

namespace dtcp {

enum GluMode { kGluForward = 0, kGluForwardE4m3 = 1, kGluBackward = 2 };

// The tiles of one product: rows x cols of output, the summed dimension `depth` (dX: of one half) in `k_iters` stages.
struct GluProduct {
  int rows, cols, depth, k_iters;
  int num_m_blocks, num_n_blocks, num_tiles, group_m;
  int split_tiles, num_items;  // trailing tiles cut into halves of their columns; work items = tiles + split_tiles
  int slices;                  // parts of the summed dimension, each an item of its own (then no halves)
  int slice_rows;              // rows from one slice's partial sums to the next one's
};

struct GluParams {
  GluProduct main;    // forward: H; backward: dX
  GluProduct second;  // backward: dWg, then dWu (rows and blocks of both)
  int ahead;          // backward: items of `second` that each cluster without a tile in dX's last wave takes meanwhile
  int act, save;
  const float* x_scale;  // E4M3: scales of X's rows, Wg's and Wu's
  const float* g_scale;
  const float* u_scale;
  unsigned* status;
  unsigned long long wait_limit_ns;
};

// One work item.
struct GluItem {
  int m_blk, n_blk, half;
  bool second;
  int slice, k0, k1;  // its stages
};

// Item `it` of a cluster; false past its last one.
__device__ __forceinline__ bool glu_item(const GluParams& p, int cluster, int clusters, int it, GluItem& item) {
  const GluProduct* q = &p.main;
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

struct GluMaps {
  CUtensorMap a0, a1;      // forward: X (both); backward: dg, du
  CUtensorMap b0, b1, b2;  // Wg, Wu; backward: X
  CUtensorMap c0, c1, c2;  // forward: H, g, u; backward: dX (or its slices' partial sums), dWg, dWu
};

// Instruction descriptor (see idesc_bf16): BF16 operands, bits 15 / 16: A / B has its M / N dimension innermost.
__host__ __device__ constexpr uint32_t idesc_glu(int m, int n, bool a_mn, bool b_mn) {
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

// An epilogue warp's staging bytes: two BF16 tiles of 32 x 32 in turn, or (`whole`) one tile, FP32 or BF16, at a time.
constexpr int kGluStagingBytes = 32 * 128;
struct GluStaging {
  uint32_t base, next;
  bool whole;
  __device__ __forceinline__ uint32_t take(uint32_t lane) {
    uint32_t buf = base;
    if (whole) {
      if (lane == 0) bulk_wait_group_read<0>();
    } else {
      buf += next * (kGluStagingBytes / 2);
      next ^= 1u;
      if (lane == 0) bulk_wait_group_read<1>();
    }
    __syncwarp();
    return buf;
  }
  __device__ __forceinline__ void store(uint32_t lane, const CUtensorMap* map, uint32_t buf, int col, int row,
                                        bool streaming) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (streaming) tma_store_2d_streaming(map, buf, col, row);
      else tma_store_2d(map, buf, col, row);
      bulk_commit_group();
    }
  }
};

// 32 columns of this lane's row as BF16 (64-byte rows, 64-byte swizzle) or FP32 (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ void glu_store(GluStaging& st, uint32_t lane, const CUtensorMap* map, const uint32_t (&v)[32],
                                          int col, int row, bool f32) {
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
  st.store(lane, map, buf, col, row, f32);
}

// The 512 x 256 pair tile (glu_wide.cu): p's products are planned for it, `clusters` pairs take them.
int glu_wide_max_clusters(int device);
int glu_wide_launch(const GluMaps& m, const GluParams& p, bool backward, int clusters, cudaStream_t stream);

}  // namespace dtcp
