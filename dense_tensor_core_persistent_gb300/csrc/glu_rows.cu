// glu_rows.cu -- the gated feed-forward block for up to 128 rows, from a single decoding sequence on:
// H = act(X Wg^T) * (X Wu^T) in BF16 or E4M3, computed as H^T so that no tensor-core row is wasted.
//
// The weights' bytes are the bound, but on the 256-row pair tile of glu.cu most of each MMA would multiply rows that
// X does not have, and under the power cap that costs clock. Here a CTA's MMA has 64 rows of Wg over 64 rows of Wu
// as its M = 128 and the rows of X as its N (a multiple of 16): accumulator lane f holds g of feature f and lane 64 + f
// its u, columns are the rows of X. The warps of the lower and of the upper lanes exchange halves of them through
// shared memory, apply the activation and the product and store 32 features of a row at a time.
//
// One persistent CTA per SM steps over tiles of 64 features; a last wave at most half full runs as halves of its
// tiles (32 features; the other accumulator lanes hold what the stage held before and are not read). Warp roles: 0
// loads W, 2 loads X, 1 allocates TMEM and issues the MMAs, 4..7 epilogue. Two accumulators in TMEM.
// Where all tiles fit at once with 2, 4 or 8 CTAs each, the CTAs of a cluster share a tile's depth: one CTA alone draws
// no more than some 50 GB/s. Each leaves its partial sums in its shared memory, and the CTAs take the rows of X in turn
// and add the cluster's sums in a fixed order.
// Measured on GB300 at 28672 x 8192 (N x K): 1 row 140 us in BF16 (6.7 TB/s of weights) and 72 in E4M3 (6.5), 64 rows
// 140 and 74 us, 128 rows 154 and 82.
// The box of X is as high as its rows need: zero rows that TMA fills in cost time too (17 rows in a box of 64 took
// 40 us in BF16 and 29 in E4M3 at 14336 x 4096, where they take 39 and 22.6 in one of 32).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "glu_act.cuh"
#include "host_common.h"

namespace dtcp {
namespace {

constexpr int kRowsMaxSplits = 8;

struct GluRowsParams {
  GluRowsOperands x;  // operands and sizes
  int k_iters, num_tiles, split_tiles, num_items;
  int splits;  // CTAs of a cluster that share a tile's depth; with more than one a cluster has one tile, and no halves
  int n;  // the MMA's N: the rows of X, rounded up to a multiple of 16
  unsigned* status;
  unsigned long long wait_limit_ns;
};

template <int X_ROWS>
struct GluRowsLayout {
  static constexpr int FEATURES = 64;
  static constexpr int ATOMS = 2;                        // 128-byte swizzle rows of K per stage
  static constexpr int KSTEPS = 4 * ATOMS;
  static constexpr int BOX_BYTES = 32 * 128;             // 32 rows of W
  static constexpr int W_ATOM_BYTES = 128 * 128, X_ATOM_BYTES = X_ROWS * 128;
  static constexpr int W_BYTES = ATOMS * W_ATOM_BYTES, X_BYTES = ATOMS * X_ATOM_BYTES;
  static constexpr int STAGES = X_ROWS == 64 ? 4 : 3;
  static constexpr int TMEM_COLS = 2 * X_ROWS;
  static constexpr int WARP_W = 0, WARP_MMA = 1, WARP_X = 2, EPI_WARP0 = 4, EPI_WARPS = 4;
  static constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int OFF_W = 0;
  static constexpr int OFF_X = STAGES * W_BYTES;
  static constexpr int OFF_U = OFF_X + STAGES * X_BYTES;  // what the epilogue exchanges: X_ROWS x FEATURES FP32
  static constexpr int OFF_BAR = OFF_U + X_ROWS * FEATURES * 4;
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;  // slack to align the base to 1024 bytes
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
};

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The epilogue's four warps meet (barrier 1).
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void store_h(const GluRowsOperands& x, int row, int f, float g, float u) {
  const float h = glu_act(g, x.act) * u;
  x.h[row * x.ldh + f] = static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(h), 0u) & 0xFFFFu);
  if (x.preact != nullptr) {
    float* pre = x.preact + static_cast<long long>(row) * 2 * x.features + f;
    pre[0] = g;
    pre[x.features] = u;
  }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

template <bool E4M3, int X_ROWS>
__global__ void __launch_bounds__(GluRowsLayout<X_ROWS>::NUM_THREADS, 1)
    glu_rows_kernel(const __grid_constant__ CUtensorMap map_g, const __grid_constant__ CUtensorMap map_u,
                    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ GluRowsParams p) {
  using L = GluRowsLayout<X_ROWS>;
  constexpr int ATOM_K = E4M3 ? 128 : 64, STAGE_K = ATOM_K * L::ATOMS, MMA_K = E4M3 ? 32 : 16;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar_full = base + L::OFF_BAR, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_tfull = bar_empty + 8 * L::STAGES, bar_tempty = bar_tfull + 16, bar_drain = bar_tempty + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_TMEM_SLOT);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + L::OFF_ABORT);
  const WaitCtx wctx{abort_flag, p.status, p.wait_limit_ns};

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(bar_full + 8 * s, 2);  // W's and X's producer
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_tfull + 8 * s, 1);
      mbar_init(bar_tempty + 8 * s, L::EPI_WARPS);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0u;
    fence_mbarrier_init_cluster();
  }
  if (warp == L::WARP_MMA) {
    tmem_alloc<1>(smem_u32(tmem_slot), L::TMEM_COLS);
    tmem_relinquish<1>();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();
  pdl_wait();
  const int splits = p.splits, rank = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / splits, step = static_cast<int>(gridDim.x) / splits;  // items
  const int k0 = rank * p.k_iters / splits, k1 = (rank + 1) * p.k_iters / splits;
  float* const partial = reinterpret_cast<float*>(smem + L::OFF_W);  // [rows of X][128]: over the stages, once they are done

  if ((warp == L::WARP_W || warp == L::WARP_X) && lane == 0) {
    // ------------------------------------------------------------ producers
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int i = first; i < p.num_items && ok; i += step) {
      const WorkItem w = work_item(i, p.num_tiles, p.split_tiles);
      const int f0 = w.tile * L::FEATURES + (w.half > 0 ? L::FEATURES / 2 : 0);
      const int boxes = w.half >= 0 ? 1 : 2;  // of 32 features
      for (int k = k0; k < k1; ++k) {
        if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
          ok = false;
          break;
        }
        const uint32_t full = bar_full + 8 * stage;
        if (warp == L::WARP_W) {
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(L::ATOMS * 2 * boxes * L::BOX_BYTES));
#pragma unroll
          for (int a = 0; a < L::ATOMS; ++a) {
            const uint32_t dst = base + L::OFF_W + stage * L::W_BYTES + a * L::W_ATOM_BYTES;
            for (int c = 0; c < boxes; ++c) {
              tma_load_2d(dst + c * L::BOX_BYTES, &map_g, k * STAGE_K + a * ATOM_K, f0 + 32 * c, full);
              tma_load_2d(dst + (2 + c) * L::BOX_BYTES, &map_u, k * STAGE_K + a * ATOM_K, f0 + 32 * c, full);
            }
          }
        } else {
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(L::ATOMS * p.n * 128));
#pragma unroll
          for (int a = 0; a < L::ATOMS; ++a)
            tma_load_2d(base + L::OFF_X + stage * L::X_BYTES + a * L::X_ATOM_BYTES, &map_x, k * STAGE_K + a * ATOM_K, 0,
                        full);
        }
        stage = stage + 1 == L::STAGES ? 0u : stage + 1;
        phase = stage == 0 ? phase ^ 1u : phase;
      }
    }
    if (!ok) settle_after_abort();
  } else if (warp == L::WARP_MMA && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    // (operand formats 0 of kind::f8f6f4 are E4M3)
    const uint32_t idesc = E4M3 ? (1u << 4) | (static_cast<uint32_t>(p.n >> 3) << 17) | ((128u >> 4) << 24)
                                : idesc_bf16(128, p.n);
    const uint64_t a0 = umma_desc_sw128(base + L::OFF_W), b0 = umma_desc_sw128(base + L::OFF_X);
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    int it = 0;
    for (int i = first; i < p.num_items && ok; i += step, ++it) {
      const uint32_t slot = static_cast<uint32_t>(it) & 1u;
      if (!wait_phase_inline(bar_tempty + 8 * slot, ((static_cast<uint32_t>(it) >> 1) & 1u) ^ 1u, wctx,
                             status_code(kRoleMma, 0x100 + slot))) {
        ok = false;
        break;
      }
      const uint32_t d = tmem_base + slot * X_ROWS;
      for (int k = k0; k < k1; ++k) {
        if (!wait_phase_inline(bar_full + 8 * stage, phase, wctx, status_code(kRoleMma, stage))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint64_t a = umma_desc_advance(a0, stage * L::W_BYTES), b = umma_desc_advance(b0, stage * L::X_BYTES);
        const int left = p.x.depth - k * STAGE_K;  // a ragged last stage: only the MMAs that hold any of it
        const int steps = left >= STAGE_K ? L::KSTEPS : (left + MMA_K - 1) / MMA_K;
        auto one = [&](int kk) {
          const uint32_t in_atom = static_cast<uint32_t>(kk % 4) * 32u, atom = static_cast<uint32_t>(kk / 4);
          const uint64_t ad = umma_desc_advance(a, atom * L::W_ATOM_BYTES + in_atom);
          const uint64_t bd = umma_desc_advance(b, atom * L::X_ATOM_BYTES + in_atom);
          if constexpr (E4M3) mma_e4m3(d, ad, bd, idesc, k != k0 || kk != 0 ? 1u : 0u);
          else mma_f16<1>(d, ad, bd, idesc, k != k0 || kk != 0 ? 1u : 0u);
        };
        if (steps == L::KSTEPS) {
#pragma unroll
          for (int kk = 0; kk < L::KSTEPS; ++kk) one(kk);
        } else {
          for (int kk = 0; kk < steps; ++kk) one(kk);
        }
        mma_commit_local(bar_empty + 8 * stage);
        stage = stage + 1 == L::STAGES ? 0u : stage + 1;
        phase = stage == 0 ? phase ^ 1u : phase;
      }
      if (ok) mma_commit_local(bar_tfull + 8 * slot);
    }
    if (!ok) {
      // let issued MMAs finish before TMEM is released (bounded: they finish or the limit passes)
      mma_commit_local(bar_drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait_suspend(bar_drain, 0, 20000u) && globaltimer_ns() - t0 < wctx.limit_ns) {
      }
      settle_after_abort();
    }
  } else if (warp >= L::EPI_WARP0) {
    // ------------------------------------------------------------ epilogue
    const uint32_t q = warp & 3u;  // TMEM lanes 32q .. 32q+31: g of features 32q.. (q < 2), u of features 32 (q - 2)..
    const bool upper = q >= 2;
    float* tile = reinterpret_cast<float*>(smem + L::OFF_U) + (q & 1u) * 32u + lane;
    bool ok = true;
    int it = 0;
    for (int i = first; i < p.num_items; i += step, ++it) {
      const WorkItem w = work_item(i, p.num_tiles, p.split_tiles);
      const int f = w.tile * L::FEATURES + (w.half > 0 ? L::FEATURES / 2 : 0) + static_cast<int>((q & 1u) * 32u + lane);
      const bool live = f < p.x.features && (w.half < 0 || (q & 1u) == 0);
      const uint32_t slot = static_cast<uint32_t>(it) & 1u;
      float g_scale = 1.0f, u_scale = 1.0f;  // E4M3: of this lane's feature, and (below) of rows of X
      if (E4M3 && live) {
        g_scale = p.x.g_scale[f];
        u_scale = p.x.u_scale[f];
      }
      if (ok)  // (after a wait that gave up the warps only keep their barriers)
        ok = wait_phase_warp(bar_tfull + 8 * slot, (static_cast<uint32_t>(it) >> 1) & 1u, wctx,
                             status_code(kRoleEpilogue, slot));
      tc_fence_after_sync();
      // Of each 32 rows of X the lower lanes' warps finish the first 16 and the upper ones' the others: a warp keeps
      // its own half of those values and leaves the other half where the other warp of its features finds it.
      const uint32_t taddr = tmem_base + ((q * 32u) << 16) + slot * X_ROWS;
      if (splits > 1) {  // every MMA of the cluster's one tile in this CTA is done
#pragma unroll 1
        for (int c = 0; 32 * c < p.x.rows; ++c) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + 32 * c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) partial[(32 * c + j) * 128 + q * 32u + lane] = __uint_as_float(v[j]);
        }
        break;
      }
      float own[X_ROWS / 32][16], xs[X_ROWS / 32];
#pragma unroll
      for (int c = 0; c < X_ROWS / 32; ++c) {
        if (32 * c >= p.x.rows) continue;
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + 32 * c, v);
        xs[c] = E4M3 && 32 * c + static_cast<int>(lane) < p.x.rows ? p.x.x_scale[32 * c + lane] : 1.0f;
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          own[c][j] = __uint_as_float(upper ? v[16 + j] : v[j]);
          tile[(32 * c + (upper ? j : 16 + j)) * L::FEATURES] = __uint_as_float(upper ? v[j] : v[16 + j]);
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_local(bar_tempty + 8 * slot);
      epilogue_sync();  // the tile is in shared memory
#pragma unroll
      for (int c = 0; c < X_ROWS / 32; ++c) {
        if (32 * c >= p.x.rows) continue;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int row = 32 * c + (upper ? 16 : 0) + j;
          const float x_scale = E4M3 ? __shfl_sync(0xffffffffu, xs[c], (upper ? 16 : 0) + j) : 1.0f;
          const float other = tile[row * L::FEATURES];
          float g = upper ? other : own[c][j], u = upper ? own[c][j] : other;
          if (E4M3) {
            g *= x_scale * g_scale;
            u *= x_scale * u_scale;
          }
          if (live && ok && row < p.x.rows) store_h(p.x, row, f, g, u);
        }
      }
      epilogue_sync();  // the tile has been read
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  if (splits > 1) {
    // The CTAs take the rows of X in turn and add the cluster's partial sums in the order of the depth.
    cluster_sync_all();
    const int f = first * L::FEATURES + static_cast<int>(threadIdx.x % L::FEATURES);
    constexpr int AT_ONCE = L::NUM_THREADS / L::FEATURES;
    if (f < p.x.features && *abort_flag == 0u) {
      const float g_scale = E4M3 ? p.x.g_scale[f] : 1.0f, u_scale = E4M3 ? p.x.u_scale[f] : 1.0f;
      for (int row = rank + splits * static_cast<int>(threadIdx.x / L::FEATURES); row < p.x.rows;
           row += splits * AT_ONCE) {
        const uint32_t at = smem_u32(partial) + (row * 128u + threadIdx.x % L::FEATURES) * 4u;
        float part[2][kRowsMaxSplits];  // asked for together
#pragma unroll
        for (int s = 0; s < kRowsMaxSplits; ++s) {
          part[0][s] = part[1][s] = 0.0f;
          if (s < splits) {
            const uint32_t from = mapa_shared(at, s);
            part[0][s] = ld_cluster_f32(from);
            part[1][s] = ld_cluster_f32(from + 4u * L::FEATURES);
          }
        }
        float g = part[0][0], u = part[1][0];
#pragma unroll
        for (int s = 1; s < kRowsMaxSplits; ++s) {
          g += part[0][s];
          u += part[1][s];
        }
        if (E4M3) {
          const float x_scale = p.x.x_scale[row];
          g *= x_scale * g_scale;
          u *= x_scale * u_scale;
        }
        store_h(p.x, row, f, g, u);
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  __syncthreads();
  if (warp == L::WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem_base, L::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side

void rows_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int grid, int threads, int smem, int splits,
                 cudaStream_t stream) {
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
}

// Prepares a kernel on a device; clusters[s]: how many clusters of 2 << s CTAs the device holds at once.
template <bool E4M3, int X_ROWS>
bool prepare_rows(int device, int (&clusters)[3]) {
  using L = GluRowsLayout<X_ROWS>;
  static std::mutex mu;
  static int cache[64][4] = {};
  std::lock_guard<std::mutex> lock(mu);
  int(&c)[4] = cache[device & 63];
  if (c[3] == 0) {
    const auto kernel = glu_rows_kernel<E4M3, X_ROWS>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_BYTES) != cudaSuccess) {
      cudaGetLastError();
      return false;
    }
    for (int s = 0; s < 3; ++s) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[2];
      rows_config(cfg, attr, 16, L::NUM_THREADS, L::SMEM_BYTES, 2 << s, nullptr);
      if (cudaOccupancyMaxActiveClusters(&c[s], kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        c[s] = 0;
      }
    }
    c[3] = 1;
  }
  for (int s = 0; s < 3; ++s) clusters[s] = c[s];
  return true;
}

template <bool E4M3, int X_ROWS>
int launch_rows(const GluRowsOperands& x, int device, const DeviceInfo* info, cudaStream_t stream) {
  using L = GluRowsLayout<X_ROWS>;
  constexpr int ATOM_K = E4M3 ? 128 : 64;
  constexpr int SIZE = E4M3 ? 1 : 2;
  const auto type = E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  GluRowsParams p;
  p.n = ceil_div(x.rows, 16) * 16;
  CUtensorMap g, u, rows;
  int st = encode_tmap_2d(&g, type, x.wg, x.depth, x.features, uint64_t(x.depth) * SIZE, ATOM_K, 32,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == GEMM_OK)
    st = encode_tmap_2d(&u, type, x.wu, x.depth, x.features, uint64_t(x.depth) * SIZE, ATOM_K, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == GEMM_OK)
    st = encode_tmap_2d(&rows, type, x.x, x.depth, x.rows, uint64_t(x.ldx) * SIZE, ATOM_K, p.n,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != GEMM_OK) return st;
  int clusters[3];
  if (!prepare_rows<E4M3, X_ROWS>(device, clusters)) return GEMM_ERR_LAUNCH;
  p.x = x;
  p.k_iters = ceil_div(x.depth, ATOM_K * L::ATOMS);
  p.num_tiles = ceil_div(x.features, L::FEATURES);
  // As many CTAs to a tile as let every tile run at once: one CTA draws at most some 50 GB/s. Measured on GB300, 1 row
  // x N x 8192 in BF16, without splits (but halves of tiles) and with the rule: N = 512 27.1 and 7.6 us (8 CTAs), 1792
  // 27.1 and 12.7 (4), 4096 28.3 and 23.7 (2); N = 5120, where two CTAs no longer fit, 33.7 and 43.4 with 2. Where the
  // sum is short the join can cost more than it saves: 128 x 4096 x 1024 in E4M3 9.4 and 10.0.
  p.splits = 1;
  for (int s = 0; s < 3; ++s)
    if (p.num_tiles <= clusters[s] && p.k_iters >= 2 << s) p.splits = 2 << s;
  p.split_tiles = p.splits > 1 ? 0 : tail_split_tiles(p.num_tiles, info->num_sms);
  p.num_items = p.num_tiles + p.split_tiles;
  p.status = device_status_word(device);
  p.wait_limit_ns = RunOptions().wait_limit_ns;
  if (p.status == nullptr) return GEMM_ERR_NO_DEVICE;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  rows_config(cfg, attr, p.splits > 1 ? p.num_items * p.splits : std::min(p.num_items, info->num_sms), L::NUM_THREADS,
              L::SMEM_BYTES, p.splits, stream);
  if (cudaLaunchKernelEx(&cfg, glu_rows_kernel<E4M3, X_ROWS>, g, u, rows, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

}  // namespace

int run_glu_rows(const GluRowsOperands& p, bool e4m3, int device, const DeviceInfo* info, cudaStream_t stream) {
  if (p.rows <= 64)
    return e4m3 ? launch_rows<true, 64>(p, device, info, stream) : launch_rows<false, 64>(p, device, info, stream);
  return e4m3 ? launch_rows<true, 128>(p, device, info, stream) : launch_rows<false, 128>(p, device, info, stream);
}

}  // namespace dtcp
