// pair_gradient.cu -- the products of a gradient on sm_103a tensor cores, dX = G W and dW = G^T X, for G in one part or in
// two ([dg | du] with [Wg ; Wu]: dX sums over both).
//
// The products need operands along their other dimension (W by columns, G and X by columns). The MMA takes them as they
// lie in memory: TMA boxes of 64 columns put the non-summed dimension innermost and the descriptors say so
// ("MN-major"), so nothing is transposed. One launch computes both: the tiles of dX, which are the longest, come first,
// and where their last wave leaves clusters free, those go ahead with as many tiles of dW as take the same time. Where
// dX has so few tiles that one would be the whole launch, their sums are cut into slices with FP32 partial sums that a
// last kernel adds in order. Where W comes in pieces, a launch each, the pieces' sums are added in memory.
//
// Bound by the tensor cores. Measured on GB300: the gated block's at 4096 x 14336 x 4096 962 to 1002 us (1.9 to 2.0
// PFLOP/s).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "host_common.h"
#include "pair_tile.cuh"

namespace dtcp {
namespace {

struct GradientParams : PairParams {
  int sums;  // dX's tiles are FP32 partial sums
  int add;   // and are added to what is in memory
};

// Where a tile goes.
struct GradientOut {
  const CUtensorMap* map;
  int m_blk, rows, cols;
  bool f32;
  PairStore how;
};
__device__ __forceinline__ GradientOut gradient_out(const GradientParams& p, const PairMaps& maps, const PairItem& item) {
  if (!item.second)
    return GradientOut{&maps.c0, item.m_blk, p.main.rows, p.main.cols, p.sums != 0, p.add ? kPairAdd : kPairPlain};
  const int part_blocks = p.second.num_m_blocks / p.parts;
  const bool last = item.m_blk >= part_blocks;
  return GradientOut{last ? &maps.c2 : &maps.c1, last ? item.m_blk - part_blocks : item.m_blk, p.second.rows,
                     p.second.cols, false, kPairPlain};
}

__global__ void __launch_bounds__(PairLayout::NUM_THREADS, 1)
    gradient_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ GradientParams p) {
  using L = PairLayout;
  pair_cta<kPairGradient>(maps, p, [&](const PairCta& c) {
    const uint32_t bar_tfull = c.base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 16;
    const uint32_t q = c.warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
    const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
    const uint32_t epi = c.warp - L::EPI_WARP0;
    const int h = static_cast<int>(epi >> 2);  // its half of the columns
    PairStaging st{c.base + L::OFF_EPI + epi * kPairStagingBytes, 0u, p.sums != 0};
    PairItem item;
    for (int it = 0; pair_item(p, c.cluster_idx, c.num_clusters, it, item); ++it) {
      const int width = item.half >= 0 ? L::BLOCK_N / 4 : L::BLOCK_N / 2;  // columns of this warp
      const int col0 = item.n_blk * L::BLOCK_N + (item.half > 0 ? 2 * width : 0) + h * width;
      const uint32_t slot = static_cast<uint32_t>(it) & 1u;
      const GradientOut o = gradient_out(p, maps, item);
      const int row0 = o.m_blk * L::TILE_M + static_cast<int>(c.rank) * L::CTA_M + static_cast<int>(q) * 32;
      if (!wait_phase_warp(bar_tfull + 8 * slot, (static_cast<uint32_t>(it) >> 1) & 1u, c.wctx,
                           status_code(kRoleEpilogue, slot)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = c.tmem_base + ((q * 32u) << 16) + slot * L::ACC_COLS + static_cast<uint32_t>(h * width);
      if (row0 < o.rows) {
#pragma unroll 1
        for (int k = 0; k < width; k += 32) {
          const int col = col0 + k;
          if (col >= o.cols) break;
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + k, v);
          tmem_ld_wait();
          pair_store(st, c.lane, o.map, v, col, row0 + item.slice * p.main.slice_rows, o.f32, o.how);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (c.lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * slot);  // orders tcgen05 work only
    }
    if (c.lane == 0) bulk_wait_group<0>();
    __syncwarp();
  });
}

__global__ void __launch_bounds__(PairWideLayout::NUM_THREADS, 1)
    gradient_wide_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ GradientParams p) {
  using L = PairWideLayout;
  pair_wide_cta<kPairGradient>(maps, p, [&](const PairCta& c) {
    const uint32_t bar_tfull = c.base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 8 * L::WAVES;
    const uint32_t q = c.warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
    const uint32_t epi = c.warp - L::EPI_WARP0;
    const int h = static_cast<int>(epi >> 2);  // its half of a wave's columns
    const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
    PairStaging st{c.base + L::OFF_EPI + epi * L::EPI_BYTES, 0u, p.sums != 0};
    bool ok = true;
    PairItem item;
    for (int it = 0; ok && pair_item(p, c.cluster_idx, c.num_clusters, it, item); ++it) {
      const int width = item.half >= 0 ? L::BLOCK_N / 4 : L::BLOCK_N / 2;  // columns of this warp
      const int col0 = item.n_blk * L::BLOCK_N + (item.half > 0 ? 2 * width : 0) + h * width;
      const GradientOut o = gradient_out(p, maps, item);
#pragma unroll 1
      for (int w = 0; w < L::WAVES; ++w) {
        const int row0 = o.m_blk * L::TILE_M + static_cast<int>(c.rank) * L::CTA_M + w * 128 + static_cast<int>(q) * 32;
        const bool live = row0 < o.rows && col0 < o.cols;
        if (!__all_sync(0xffffffffu, wait_phase_inline(bar_tfull + 8 * w, static_cast<uint32_t>(it) & 1u, c.wctx,
                                                       status_code(kRoleEpilogue, w)))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t taddr = c.tmem_base + ((q * 32u) << 16) + static_cast<uint32_t>(w) * L::ACC_COLS +
                               static_cast<uint32_t>(h * width);
        uint32_t v[4][32];
        if (live) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k * 32 < width) tmem_ld_32x32b_x32(taddr + k * 32, v[k]);
          tmem_ld_wait();
        }
        // the wave's columns are read: hand them back to the MMA issuer (leader's barrier)
        tc_fence_before_sync();
        __syncwarp();
        if (c.lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * w);  // orders tcgen05 work only
        if (!live) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k * 32 < width && col0 + k * 32 < o.cols)
            pair_store(st, c.lane, o.map, v[k], col0 + k * 32, row0, o.f32, o.how);
      }
    }
    if (c.lane == 0) bulk_wait_group<0>();
    __syncwarp();
  });
}

// ---------------------------------------------------------------- dX from its slices

// The sum of the slices' partial sums in their order, rounded once: 8 columns per thread. `half`: each slice has a second
// part of the rows that far behind the first (0: none).
__global__ void __launch_bounds__(128) join_kernel(const float* partial, int slices, long long slice_size, long long half,
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
    if (half > 0) {
      const float4 a = *reinterpret_cast<const float4*>(at + s * slice_size + half);
      const float4 b = *reinterpret_cast<const float4*>(at + s * slice_size + half + 4);
      const float f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j] += f[j];
    }
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

int gradient_max_clusters(int device, bool wide) {
  static std::mutex mu;
  static int cache[64][2] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  int& n = cache[device][wide ? 1 : 0];
  if (n == 0) {
    const void* kernel = wide ? reinterpret_cast<const void*>(gradient_wide_kernel)
                              : reinterpret_cast<const void*>(gradient_kernel);
    n = pair_max_clusters(&kernel, 1, wide);
  }
  return n;
}

// Parts of dX's summed dimension, where its few tiles would be the launch's longest path: the stages of a tile against
// the stages of all tiles of both products spread over the pairs (with two more for a short tile of dW's end). A part
// has 6 stages at least, the parts run at once, and what is saved has to pay for the partial sums and the kernel that
// adds them, some 4 us (8 stages). Measured on GB300, whole gradient: 512 x 4096 x 1024 44.2 us in one part and 24.3 in
// four, 300 x 1368 x 520 22.3 and 17.3 in three; 10 x 2072 x 5576, which stays whole, 30.2 and 33.0 in three.
int gradient_slices(const PairProduct& dx, const PairProduct& dw, int wave) {
  const long long work = 1LL * dx.num_tiles * dx.k_iters + 1LL * dw.num_tiles * (dw.k_iters + 2);
  const int share = std::max<int>(6, static_cast<int>(std::min<long long>(work / wave, 0x7FFFFFFF)));
  const int slices = std::min({8, dx.k_iters / share, wave / dx.num_tiles});
  return slices > 1 && dx.k_iters - dx.k_iters / slices >= 12 ? slices : 1;
}

// What a tile of dW costs, in stages: a shallow one is bound by its store (64 rows x 32768 x 4096: 2.1 us a tile, where a
// stage of dX takes 0.85).
double shallow_cost(const PairProduct& dw) { return std::max<double>(dw.k_iters, 2.5); }

// The same where the features are a piece of a large vocabulary: as many parts as bring a tile of dX within a twelfth of an
// even share of the launch. Measured on GB300, whole gradient of the cross entropy, by parts (in parentheses a whole tile in
// shares): 64 x 131072 x 4096 876 us in one, 638, 608, 582 in two to four (2.1); 700 x 50000 x 776 317 in one, 206, 166, 171
// in two to four (3.2); 200 x 131072 x 1024 391, 254, 210, 190, 195 in two, four, six, eight, twelve (8.4); 128 x 8192 x
// 8192, which stays whole, 99 and 105 in two (1.06). Without dW nothing else fills a last round of parts, so their rounds
// count: 64 x 131072 x 4096 439 us in five and 348 in nine, 700 x 50000 x 776 145 in seven and 116 in six.
int gradient_slices_even(const PairProduct& dx, const PairProduct& dw, int wave) {
  if (dw.num_tiles == 0) {
    auto rounds = [&](int s) { return ceil_div(dx.num_tiles * s, wave) * (ceil_div(dx.k_iters, s) + 3); };
    int best = 1;
    if (dx.num_tiles < wave)
      for (int s = 2; s <= 16 && dx.k_iters / s >= 6; ++s)
        if (rounds(s) + 2 * s < rounds(best) + 2 * best) best = s;
    return best;
  }
  const double share = (1.0 * dx.num_tiles * dx.k_iters + dw.num_tiles * shallow_cost(dw)) / wave;
  const int slices = static_cast<int>(dx.k_iters / std::max(share, 6.0) + 0.92);
  return std::max(1, std::min(slices, 16));
}

// The order of a product's tiles on `clusters` pairs, for operands of `bytes` per element.
void order_product(PairProduct* q, int clusters, int tile_rows, double bytes, long long l2_bytes) {
  constexpr int BLOCK_N = PairLayout::BLOCK_N;
  q->group_m = choose_group_m(static_cast<int>(std::min<long long>(1LL * q->num_m_blocks * tile_rows, 0x7FFFFFFF)),
                              static_cast<int>(std::min<long long>(1LL * q->num_n_blocks * BLOCK_N, 0x7FFFFFFF)),
                              std::max(q->depth, 1), tile_rows, BLOCK_N, bytes, 0.0, clusters, l2_bytes);
}

}  // namespace

bool pair_gradient_is_wide(const PairGradient& q, int wave) {
  using L = PairLayout;
  const bool dx = q.dx != nullptr, dw = q.dw[0] != nullptr;
  const int M = q.rows, N = q.features[0], parts = q.parts;
  if (M == 0) return false;
  // in tiles of dW (their depth is M), of which one of dX (its depth is all features) counts several
  const double long_tile = dw ? 1.0 * parts * N / M : 1.0;
  const long long k_tiles = ceil_div(q.K, L::BLOCK_N);
  auto tiles = [&](int tile_rows) {
    return static_cast<long long>(dx ? long_tile * ceil_div(M, tile_rows) * k_tiles : 0.0) +
           (dw ? 1LL * parts * ceil_div(N, tile_rows) * k_tiles : 0LL);
  };
  const int depth =
      !dw ? static_cast<int>(std::min(1LL * parts * N, 0x7FFFFFFFLL)) : !dx ? M : std::min(M, N);
  return pair_wide_rule(tiles(L::TILE_M), tiles(2 * L::TILE_M), depth, wave);
}

int pair_max_clusters(const void* const* kernels, int count, bool wide) {
  const int smem = wide ? PairWideLayout::SMEM_BYTES : PairLayout::SMEM_BYTES;
  for (int i = 0; i < count; ++i)
    if (cudaFuncSetAttribute(kernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(2 * 16, 1, 1);
  cfg.blockDim = dim3(wide ? PairWideLayout::NUM_THREADS : PairLayout::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernels[0], &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

int pair_map_in(CUtensorMap* m, const void* p, int cols, int rows, long long ld, int box_rows) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, rows, uint64_t(ld) * 2, 64, box_rows,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}
int pair_map_out(CUtensorMap* m, const void* p, int cols, int rows, long long ld) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, cols, rows, uint64_t(ld) * 2, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_64B);
}
int pair_map_out_f32(CUtensorMap* m, const void* p, int cols, uint64_t rows, long long ld) {
  return encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p, cols, rows, uint64_t(ld) * 4, 32, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

int pair_plan_product(PairProduct* q, int rows, int cols, int depth, int stage, int parts, int outputs, int tile_rows,
                      int cols_a_tile) {
  q->rows = rows;
  q->cols = cols;
  q->depth = depth;
  q->k_iters = parts * ceil_div(depth, stage);
  const long long m = static_cast<long long>(outputs) * ceil_div(rows, tile_rows);
  q->num_n_blocks = ceil_div(cols, cols_a_tile);
  if (m * q->num_n_blocks > 0x1FFFFFFFLL) return GEMM_ERR_UNSUPPORTED_SHAPE;
  q->num_m_blocks = static_cast<int>(m);
  q->num_tiles = q->num_items = static_cast<int>(m * q->num_n_blocks);
  q->split_tiles = 0;
  q->slices = 1;
  return GEMM_OK;
}

// The 512 x 256 pair tile moves a quarter fewer bytes from L2 per operation but has half the tiles and one accumulator, so
// it needs a deep sum and is taken where the launch, in tile-times of the 256 x 256 tile, is shorter with wide tiles at
// 2 / 1.06 each: 1.06 is its gain per unit of work. Measured on GB300 on 64 shapes from 2048 deep on whose two estimates
// are within 12%: rows of X that start on 128-byte boundaries show 1.03 in the mean, forward (0.98 to 1.07: 178 us on the
// 256 x 256 tile and 174 on this one at 5951 x 3904 x 3264, 115 and 118 at 3853 x 5504 x 2176) and in the gradient (0.94 to
// 1.14); other rows 1.13 and 1.11 (352 and 300 us at 9034 x 5016 x 2744). The rule is 0.6% and 1.5% slower in the mean
// than the better tile of each shape on the former, 4% and 2% on the latter.
bool pair_wide_rule(long long std_tiles, long long wide_tiles, int depth, int wave) {
  return depth >= 2048 && 2.0 * launch_tile_times(wide_tiles, wave) / 1.06 < launch_tile_times(std_tiles, wave);
}

int pair_schedule(PairParams* p, bool wide, double bytes, int wave, int device, const DeviceInfo* info, bool even) {
  using L = PairLayout;
  p->status = device_status_word(device);
  p->wait_limit_ns = RunOptions().wait_limit_ns;
  if (p->status == nullptr) return -GEMM_ERR_NO_DEVICE;
  PairProduct &a = p->main, &b = p->second;
  p->ahead = 0;
  if (b.num_tiles == 0 && a.slices == 1) {
    a.split_tiles = tail_split_tiles(a.num_tiles, wave);
    a.num_items = a.num_tiles + a.split_tiles;
  } else if (b.num_tiles > 0) {
    // clusters that a last partial wave of the first product leaves free go ahead with tiles of the second
    const int clusters = std::min(a.num_items + b.num_tiles, wave);
    const int in_last = a.num_items % clusters, idle = in_last > 0 ? clusters - in_last : 0;
    if (idle > 0)
      p->ahead = std::min(even ? static_cast<int>(a.k_iters / a.slices / shallow_cost(b))
                               : (a.k_iters / a.slices + b.k_iters / 2) / b.k_iters,
                          ceil_div(b.num_tiles, idle));
    const int rest = std::max(0, b.num_tiles - p->ahead * idle);
    b.split_tiles = tail_split_tiles(rest, wave);
    b.num_items = b.num_tiles + b.split_tiles;
  }
  const int clusters = std::min(a.num_items + b.num_items, wave);
  const int tile_rows = wide ? 2 * L::TILE_M : L::TILE_M;
  order_product(&a, clusters, tile_rows, bytes, info->l2_bytes);
  if (b.num_tiles > 0) order_product(&b, clusters, tile_rows, bytes, info->l2_bytes);
  // dW of a large vocabulary: whole rows of it next to one another in time, which memory takes better, as soon as X's rows,
  // that its tiles share, stay in L2 anyway. Measured on GB300, whole gradient of the cross entropy, with the order for
  // operands from memory and with this: 64 x 131072 x 4096 590 and 567 us, 1000 x 64000 x 2048 505 and 447, 700 x 50000 x
  // 776 169 and 157; from 2000 rows on the same.
  if (even && b.num_tiles > 0) b.group_m = 4;
  return clusters;
}

int pair_launch(const void* kernel, void** args, bool wide, int clusters, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2), 1, 1);
  cfg.blockDim = dim3(wide ? PairWideLayout::NUM_THREADS : PairLayout::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = wide ? PairWideLayout::SMEM_BYTES : PairLayout::SMEM_BYTES;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

int pair_gradient_plan(const PairGradient& q, int device, PairGradientPlan* plan) {
  using L = PairLayout;
  const int wave = gradient_max_clusters(device, false);
  if (wave <= 0) return GEMM_ERR_LAUNCH;
  *plan = PairGradientPlan{};
  PairParams& p = plan->p;
  p.parts = q.parts;
  p.main.slices = p.second.slices = 1;
  plan->wide = pair_gradient_is_wide(q, wave);
  const int stage = plan->wide ? 64 : 128, tile_rows = plan->wide ? 2 * L::TILE_M : L::TILE_M;
  int st = GEMM_OK;
  if (q.dx != nullptr)
    st = pair_plan_product(&p.main, q.rows, q.K, q.features[0], stage, q.parts, 1, tile_rows, L::BLOCK_N);
  if (st == GEMM_OK && q.dw[0] != nullptr)
    st = pair_plan_product(&p.second, q.features[0], q.K, q.rows, stage, 1, q.parts, tile_rows, L::BLOCK_N);
  if (st != GEMM_OK) return st;
  if (q.dx != nullptr) {
    if (!plan->wide)
      p.main.slices = q.even ? gradient_slices_even(p.main, p.second, wave) : gradient_slices(p.main, p.second, wave);
    if (q.most_slices > 0) p.main.slices = std::min(p.main.slices, q.most_slices);
    p.main.num_items = p.main.num_tiles * p.main.slices;
    p.main.slice_rows = ceil_div(q.rows, 32) * 32;
    if (p.main.slices > 1 || q.keep_sums) plan->sums = size_t(p.main.slices) * p.main.slice_rows * q.K;
  }
  return GEMM_OK;
}

int pair_gradient_launch(const PairGradient& q, PairGradientPlan* plan, float* sums, int device, const DeviceInfo* info,
                         cudaStream_t stream) {
  GradientParams p;
  static_cast<PairParams&>(p) = plan->p;
  p.sums = plan->sums > 0 ? 1 : 0;
  p.add = q.add ? 1 : 0;
  const int stage = plan->wide ? 64 : 128, last = q.parts - 1;
  PairMaps m;
  // (a box of 64 features is the same for either order)
  int st = pair_map_in(&m.a0, q.g[0], q.features[0], q.rows, q.ldg, stage);
  if (st == GEMM_OK) st = pair_map_in(&m.a1, q.g[last], q.features[last], q.rows, q.ldg, stage);
  m.b0 = m.b1 = m.b2 = m.c0 = m.c1 = m.c2 = m.a0;
  if (q.dx != nullptr) {
    if (st == GEMM_OK) st = pair_map_in(&m.b0, q.w[0], q.K, q.features[0], q.K, stage);
    if (st == GEMM_OK) st = pair_map_in(&m.b1, q.w[last], q.K, q.features[last], q.K, stage);
    if (st == GEMM_OK)
      st = p.sums ? pair_map_out_f32(&m.c0, sums, q.K, uint64_t(p.main.slices) * p.main.slice_rows, q.K)
                  : pair_map_out(&m.c0, q.dx, q.K, q.rows, q.lddx);
  }
  if (q.dw[0] != nullptr) {
    if (st == GEMM_OK) st = pair_map_in(&m.b2, q.x, q.K, q.rows, q.ldx, stage);
    if (st == GEMM_OK) st = pair_map_out(&m.c1, q.dw[0], q.K, q.features[0], q.K);
    if (st == GEMM_OK) st = pair_map_out(&m.c2, q.dw[last], q.K, q.features[last], q.K);
  }
  if (st != GEMM_OK) return st;
  const int wave = gradient_max_clusters(device, plan->wide);
  if (wave <= 0) return GEMM_ERR_LAUNCH;
  const int clusters = pair_schedule(&p, plan->wide, 2.0, wave, device, info, q.even);
  if (clusters < 0) return -clusters;
  void* args[] = {&m, &p};
  return pair_launch(plan->wide ? reinterpret_cast<const void*>(gradient_wide_kernel)
                                : reinterpret_cast<const void*>(gradient_kernel),
                     args, plan->wide, clusters, stream);
}

int pair_gradient_join(const float* sums, int slices, void* dx, long long lddx, int rows, int K, cudaStream_t stream,
                       bool halves) {
  const long long vectors = static_cast<long long>(rows) * (K / 8);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>((vectors + 127) / 128), 1, 1);
  cfg.blockDim = dim3(128, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const long long slice_size = static_cast<long long>(ceil_div(halves ? 2 * rows : rows, 32)) * 32 * K;
  const long long half = halves ? static_cast<long long>(rows) * K : 0;
  if (cudaLaunchKernelEx(&cfg, join_kernel, sums, slices, slice_size, half, static_cast<uint16_t*>(dx), lddx, K, vectors) !=
      cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

}  // namespace dtcp
