// glu.cu -- the gated feed-forward block H = act(X Wg^T) * (X Wu^T) on sm_103a tensor cores, its
// form with E4M3 operands and a scale per row, and its gradient.
//
//   g = X Wg^T, u = X Wu^T (M x N, FP32),  H = act(g) u
//   dg = dH u act'(g), du = dH act(g),  dX = dg Wg + du Wu,  dWg = dg^T X,  dWu = du^T X
//
// A persistent, warp-specialised kernel on a 256 x 256 tile per CTA pair (pair_tile.cuh; cta_group::2 MMAs, M = 256,
// N = 256, FP32 accumulators, two of them in TMEM): A = X and B = 128 rows of Wg (the pair's first CTA loads them) over
// 128 rows of Wu (the second one), so columns 0..127 of the accumulator are g and columns 128..255 are u of the same
// features, and the epilogue has both in one TMEM lane: both projections, the activation and the product are one
// kernel, and X is read once for the two. The gradient's products are pair_gradient.cu's, from [dg | du] and
// [Wg ; Wu].
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
namespace {

template <int MODE>
__global__ void __launch_bounds__(PairLayout::NUM_THREADS, 1)
    glu_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ GluParams p) {
  using L = PairLayout;
  pair_cta<MODE>(maps, p, [&](const PairCta& c) {
    const uint32_t bar_tfull = c.base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 16;
    const uint32_t q = c.warp & 3u;  // this warp may access TMEM lanes 32q .. 32q+31
    const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
    const uint32_t epi = c.warp - L::EPI_WARP0;
    const int h = static_cast<int>(epi >> 2);  // its half of the columns
    const int rows = p.main.rows, cols = p.main.cols;
    PairStaging st{c.base + L::OFF_EPI + epi * kPairStagingBytes, 0u, p.save != 0};
    PairItem item;
    for (int it = 0; pair_item(p, c.cluster_idx, c.num_clusters, it, item); ++it) {
      const int columns = item.half >= 0 ? L::BLOCK_N / 2 : L::BLOCK_N;  // of the item's accumulator
      const int width = columns / 4;                                     // features of this warp: 64 or 32
      const int col0 = item.n_blk * L::FEATURES + (item.half > 0 ? 2 * width : 0) + h * width;
      const uint32_t slot = static_cast<uint32_t>(it) & 1u;
      const int row0 = item.m_blk * L::TILE_M + static_cast<int>(c.rank) * L::CTA_M + static_cast<int>(q) * 32;
      // E4M3: this lane's row scale and its features' scales, while the MMAs run
      float x_scale = 1.0f, w_scale[2][L::FEATURES / 64];
      if constexpr (MODE == kPairGatedE4m3) {
        if (row0 + static_cast<int>(c.lane) < rows) x_scale = p.x_scale[row0 + c.lane];
#pragma unroll
        for (int k = 0; k < L::FEATURES / 64; ++k) {
          const int f = col0 + k * 32 + static_cast<int>(c.lane);
          w_scale[0][k] = f < cols ? p.g_scale[f] : 0.0f;
          w_scale[1][k] = f < cols ? p.u_scale[f] : 0.0f;
        }
      }
      if (!wait_phase_warp(bar_tfull + 8 * slot, (static_cast<uint32_t>(it) >> 1) & 1u, c.wctx,
                           status_code(kRoleEpilogue, slot)))
        break;
      tc_fence_after_sync();
      const uint32_t taddr = c.tmem_base + ((q * 32u) << 16) + slot * L::ACC_COLS + static_cast<uint32_t>(h * width);
      if (row0 < rows) {
        const float xs = x_scale;
#pragma unroll MODE == kPairGatedE4m3 ? 2 : 1
      for (int k = 0; k < L::FEATURES / 2; k += 32) {
        const int col = col0 + k;
        if (k >= width || col >= cols) break;
        float gs = 0.0f, us = 0.0f;  // E4M3: the scales of feature col + lane
        if constexpr (MODE == kPairGatedE4m3) {
          gs = w_scale[0][k / 32];
          us = w_scale[1][k / 32];
        }
        uint32_t g[32], u[32];
        tmem_ld_32x32b_x32(taddr + k, g);
        tmem_ld_32x32b_x32(taddr + columns / 2 + k, u);
        tmem_ld_wait();
        if (p.save) {
          pair_store(st, c.lane, &maps.c1, g, col, row0, true, kPairStreaming);
          pair_store(st, c.lane, &maps.c2, u, col, row0, true, kPairStreaming);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float gv = __uint_as_float(g[j]), uv = __uint_as_float(u[j]);
          if constexpr (MODE == kPairGatedE4m3) {
            gv *= xs * __shfl_sync(0xffffffffu, gs, j);
            uv *= xs * __shfl_sync(0xffffffffu, us, j);
          }
          g[j] = __float_as_uint(glu_act(gv, p.act) * uv);
        }
        pair_store(st, c.lane, &maps.c0, g, col, row0, false);
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

// ---------------------------------------------------------------- host side

int glu_max_clusters(int device) {
  static std::mutex mu;
  static int cache[64] = {0};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  if (cache[device] == 0) {
    const void* kernels[] = {reinterpret_cast<const void*>(glu_kernel<kPairGated>),
                             reinterpret_cast<const void*>(glu_kernel<kPairGatedE4m3>)};
    cache[device] = pair_max_clusters(kernels, 2, false);
  }
  return cache[device];
}

template <int MODE>
int glu_launch(const PairMaps& m, GluParams& p, bool wide, double bytes, int device, const DeviceInfo* info,
               cudaStream_t stream) {
  const int wave = wide ? glu_wide_max_clusters(device) : glu_max_clusters(device);
  if (wave <= 0) return GEMM_ERR_LAUNCH;
  const int clusters = pair_schedule(&p, wide, bytes, wave, device, info);
  if (clusters < 0) return -clusters;
  if (wide) return glu_wide_launch(m, p, clusters, stream);
  void* args[] = {const_cast<PairMaps*>(&m), &p};
  return pair_launch(reinterpret_cast<const void*>(glu_kernel<MODE>), args, false, clusters, stream);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool glu_forward_wide(int M, int N, int K, int wave) {
  using L = PairLayout;
  const long long n_tiles = ceil_div(N, L::FEATURES);
  return pair_wide_rule(ceil_div(M, L::TILE_M) * n_tiles, ceil_div(M, 2 * L::TILE_M) * n_tiles, K, wave);
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
  PairGradient q = {};
  q.dx = q.dw[0] = forward;  // (all gradients; nothing is read)
  q.rows = M;
  q.features[0] = q.features[1] = N;
  q.K = K;
  q.parts = 2;
  *backward = pair_gradient_is_wide(q, wave) ? 512 : 256;
  return GEMM_OK;
}

int gemm_glu_bf16(const void* X, const void* Wg, const void* Wu, void* H, float* preact, int M, int N, int K, int act,
                  void* stream, const gemm_glu_strides_t* strides) {
  using L = PairLayout;
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
  PairMaps m;
  GluParams p = {};
  const bool wide = glu_forward_wide(M, N, K, glu_max_clusters(device));
  int st = pair_map_in(&m.a0, X, K, M, ld.x, wide ? 64 : 128);
  if (st == GEMM_OK) st = pair_map_in(&m.b0, Wg, K, N, K, 64);  // (half its rows: a half tile's load is one box)
  if (st == GEMM_OK) st = pair_map_in(&m.b1, Wu, K, N, K, 64);
  if (st == GEMM_OK) st = pair_map_out(&m.c0, H, N, M, ld.h);
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
  st = pair_plan_product(&p.main, M, N, K, wide ? 64 : 128, 1, 1, wide ? 2 * L::TILE_M : L::TILE_M, L::FEATURES);
  return st != GEMM_OK ? st : glu_launch<kPairGated>(m, p, wide, 2.0, device, info, s);
}

int gemm_glu_e4m3(const void* X, const float* x_scale, const void* Wg, const float* wg_scale, const void* Wu,
                  const float* wu_scale, void* H, int M, int N, int K, int act, void* stream,
                  const gemm_glu_strides_t* strides) {
  using L = PairLayout;
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
  PairMaps m;
  GluParams p = {};
  auto map8 = [&](CUtensorMap* t, const void* q, int rows, long long stride, int box_rows) {
    return encode_tmap_2d(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, K, rows, stride, 128, box_rows,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  };
  int st = map8(&m.a0, X, M, ld.x, 128);
  if (st == GEMM_OK) st = map8(&m.b0, Wg, N, K, 64);
  if (st == GEMM_OK) st = map8(&m.b1, Wu, N, K, 64);
  if (st == GEMM_OK) st = pair_map_out(&m.c0, H, N, M, ld.h);
  if (st != GEMM_OK) return st;
  m.a1 = m.b2 = m.a0;
  m.c1 = m.c2 = m.c0;
  p.act = act;
  p.x_scale = x_scale;
  p.g_scale = wg_scale;
  p.u_scale = wu_scale;
  st = pair_plan_product(&p.main, M, N, K, 256, 1, 1, L::TILE_M, L::FEATURES);
  return st != GEMM_OK ? st : glu_launch<kPairGatedE4m3>(m, p, false, 1.0, device, info, s);
}

int gemm_glu_bf16_backward(const void* dH, const void* X, const void* Wg, const void* Wu, const float* preact, void* dX,
                           void* dWg, void* dWu, int M, int N, int K, int act, void* stream,
                           const gemm_glu_strides_t* strides) {
  using L = PairLayout;
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
  PairGradient q = {};
  q.x = X;
  q.w[0] = Wg;
  q.w[1] = Wu;
  q.dx = dX;
  q.dw[0] = dWg;
  q.dw[1] = dWu;
  q.ldg = 2LL * N;
  q.ldx = ld.x;
  q.lddx = ld.dx;
  q.rows = M;
  q.features[0] = q.features[1] = N;
  q.K = K;
  q.parts = 2;
  PairGradientPlan plan;
  int st = pair_gradient_plan(q, device, &plan);
  if (st != GEMM_OK) return st;
  const size_t gate_bytes = size_t(M) * N * 4;  // N % 8 == 0: the partial sums start on a 16-byte boundary
  cudaMemPool_t pool = workspace_pool(device);
  void* ws = nullptr;
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, gate_bytes + plan.sums * 4, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  float* const sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + gate_bytes);
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
  q.g[0] = dgu;
  q.g[1] = dgu + N;
  if (st == GEMM_OK) st = pair_gradient_launch(q, &plan, sums, device, info, s);
  if (st == GEMM_OK && plan.sums > 0) st = pair_gradient_join(sums, plan.p.main.slices, dX, ld.dx, M, K, s);
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

}  // extern "C"
