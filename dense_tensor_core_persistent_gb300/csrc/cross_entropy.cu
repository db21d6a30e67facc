// cross_entropy.cu -- softmax cross entropy of the head's logits against given targets, and its gradient, without
// storing the logits:
//
//   z = X W^T (M x V, FP32),  lse = log sum_j exp(scale z_j),  loss = lse - scale z_target
//   G = scale ((dloss + dlse) p - dloss 1[target]),  p_j = exp(scale z_j - lse),  dX = G W,  dW = G^T X
//
// Forward: the products run on the pair tiles of pair_tile.cuh, and the epilogue reduces a row's 128 (or 64) columns of
// a tile to their maximum m, the sum of exp(z - m) over the others, and the target's logit where it is among them. A
// second kernel joins a row's parts in a fixed order. The maximum's own term is exactly 1 and is kept out of the sums,
// so lse and loss end in log1p and a row that its target dominates keeps its digits.
//
// Gradient: for a piece of the vocabulary at a time the logits are computed again, in the same parts of their depth as the
// forward pass, their epilogue turns them into G (BF16, the operand of two products) and pair_gradient.cu's launch takes G to
// the piece's rows of dW and to dX, whose pieces are added in FP32. A piece is as large as G's workspace may be; fewer pieces
// are fewer joins and ramps. Not keeping z costs its product a second time: 8 MVK operations where 6 would do with M x V
// logits in memory. (Up to 64 rows G comes from cross_entropy_rows.cu: 30 x 100000 x 2048 286 us with the pair tile, 242 so.)
//
// G's rounding is seen: dX and dW are 2.4e-3 of their size from 64 bits, where their own rounding to BF16 alone leaves 1.7e-3.
// A second BF16 number for what the first one's rounding left would take that away, at 4 MVK operations more on top of the 8
// of both passes (TF32 operands, at half the rate, cost the same). So above 64 rows it is one number.
//
// Bound by the tensor cores, for few rows by W's bytes. Measured on GB300: 4096 x 131072 x 4096 forward 2.24 ms (1.96
// PFLOP/s), gradient 7.5 ms on a cool device (1.76 PFLOP/s over its three products; with one accumulator for the logits' depth
// 7.4) and up to 8.0 ms under the power cap; 4096 x 32768 x 1024 154 and 500 us; 64 x 131072 x 4096 gradient 579 us, where
// reading W twice and writing dW takes 475.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "loss_common.cuh"
#include "pair_tile.cuh"

namespace dtcp {
namespace {

constexpr size_t kLossWorkspace = size_t(512) << 20;  // bytes of G at a time, where the caller gives no limit

struct LossParams : PairParams {
  float scale;
  const long long* targets;  // or null
  int first_col;             // the piece's first column
  int vocab;
  // forward
  float2* parts;     // [blocks of 256 columns][2][rows]: (m, sum of the others)
  float2* extra;     // [tiles cut in halves][2][rows of a tile]: the second 64 columns of a half
  float* target_z;   // [rows]
  LossGradient grad;
};

// The place of a tile in its product's order.
__device__ __forceinline__ int tile_index(const PairProduct& q, int m_blk, int n_blk) {
  const int group_m = min(q.group_m, q.num_m_blocks);
  const int g = m_blk / group_m, first = g * group_m, rows = min(q.num_m_blocks - first, group_m);
  return g * group_m * q.num_n_blocks + n_blk * rows + m_blk - first;
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 32 columns of a row, of which the first `valid` exist. A knockout leaves the maximum and its 31 losers, ties among them,
// so that no element has to be told from the maximum. (v is used up.)
__device__ __forceinline__ SoftmaxPart part_of(float (&v)[32], int valid, float c) {
  if (valid < 32) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j >= valid) v[j] = -INFINITY;
  }
#pragma unroll
  for (int n = 16; n > 0; n >>= 1) {
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float a = v[j], b = v[j + n];
      v[j] = max_nan(a, b);
      v[j + n] = min_nan(a, b);
    }
  }
  const float m = v[0];
  const uint64_t off = f2_pack(-m, -m), c2 = f2_pack(c, c);
  uint64_t sum[2] = {0, 0};
  float e0, e1;
#pragma unroll
  for (int j = 2; j < 32; j += 2) {
    f2_unpack(f2_mul(f2_add(f2_pack(v[j], v[j + 1]), off), c2), e0, e1);
    sum[(j >> 1) & 1] = f2_add(sum[(j >> 1) & 1], f2_pack(ex2_approx(e0), ex2_approx(e1)));
  }
  f2_unpack(f2_add(sum[0], sum[1]), e0, e1);
  const float others = ex2_approx((v[1] - m) * c) + (e0 + e1);
  return SoftmaxPart{m, m == -INFINITY ? 0.0f : others};
}

__device__ __forceinline__ float pick(const float (&v)[32], int i) {
  float r = v[0];
#pragma unroll
  for (int j = 1; j < 32; ++j) r = i == j ? v[j] : r;
  return r;
}

// One row of the forward epilogue: chunks of 32 columns, then where the result goes.
struct LossRow {
  long long target;  // -1: none
  SoftmaxPart part;
  float c;
  __device__ __forceinline__ void begin(const LossParams& p, int row) {
    target = p.targets != nullptr && row < p.main.rows ? p.targets[row] : -1;
    part = SoftmaxPart{-INFINITY, -1.0f};  // an empty set: joined to another it adds (-1 + 1) exp(-inf) = 0
    c = log2_scale(p.scale);
  }
  __device__ __forceinline__ void chunk(const LossParams& p, float (&v)[32], int row, int col) {
    const long long t = target - col;
    if (t >= 0 && t < 32 && target < p.vocab) p.target_z[row] = pick(v, static_cast<int>(t));
    part = join(part_of(v, p.main.cols - col, c), part, c);
  }
  __device__ __forceinline__ void end(const LossParams& p, const PairItem& item, int h, int row) {
    if (row >= p.main.rows) return;
    float2* to = p.parts + (static_cast<long long>(item.n_blk) * 2 + (item.half < 0 ? h : item.half)) * p.main.rows + row;
    if (item.half >= 0 && h == 1) {
      const int i = tile_index(p.main, item.m_blk, item.n_blk) - (p.main.num_tiles - p.main.split_tiles);
      constexpr int TILE_M = PairLayout::TILE_M;
      to = p.extra + (static_cast<long long>(i) * 2 + item.half) * TILE_M + (row - item.m_blk * TILE_M);
    }
    *to = make_float2(part.m, part.others);
  }
};

// One row of the gradient's epilogue: logits become G.
struct GradRow {
  GradientRow g;
  float scale;
  __device__ __forceinline__ void begin(const LossParams& p, int row) {
    g = GradientRow(p.grad, row);
    scale = p.scale;
  }
  __device__ __forceinline__ void chunk(uint32_t (&v)[32], int col) const {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      v[j] = __float_as_uint(gradient_of(__uint_as_float(v[j]), scale, g.lse, g.softmax, g.dead));
    const long long t = g.target - col;
    if (t >= 0 && t < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (t == j) v[j] = __float_as_uint(__uint_as_float(v[j]) - g.onehot);
    }
  }
};

// An epilogue warp's 128 columns of a tile (64 of a half), added over the parts of the depth; false if a wait ran out. An
// accumulator goes back to the MMAs as soon as it is read.
__device__ __forceinline__ bool add_parts(const PairCta& c, int parts, int width, bool live, uint32_t& acc,
                                          float (&sum)[4][32]) {
  using L = PairLayout;
  const uint32_t bar_tfull = c.base + L::OFF_BAR + 16 * L::STAGES, bar_tempty = bar_tfull + 16;
  const uint32_t q = c.warp & 3u, h = (c.warp - L::EPI_WARP0) >> 2;
  const uint32_t tempty_leader = mapa_shared(bar_tempty, 0);
#pragma unroll 1
  for (int part = 0; part < parts; ++part, ++acc) {
    const uint32_t slot = acc & 1u;
    if (!__all_sync(0xffffffffu, wait_phase_inline(bar_tfull + 8 * slot, (acc >> 1) & 1u, c.wctx,
                                                   status_code(kRoleEpilogue, slot))))
      return false;
    tc_fence_after_sync();
    if (live) {
      const uint32_t taddr =
          c.tmem_base + ((q * 32u) << 16) + slot * L::ACC_COLS + h * static_cast<uint32_t>(width);
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        if (k * 32 >= width) continue;
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(taddr + k * 32, v[0]);
        tmem_ld_32x32b_x32(taddr + k * 32 + 32, v[1]);
        tmem_ld_wait();
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            sum[k + t][j] = part == 0 ? __uint_as_float(v[t][j]) : sum[k + t][j] + __uint_as_float(v[t][j]);
      }
    }
    tc_fence_before_sync();
    __syncwarp();
    if (c.lane == 0) mbar_arrive_cluster_relaxed(tempty_leader + 8 * slot);  // orders tcgen05 work only
  }
  return true;
}

// The rows and columns of an epilogue warp in a tile.
struct LossPlace {
  int width, col0, row0, row;
  bool live;
  __device__ __forceinline__ LossPlace(const LossParams& p, const PairCta& c, const PairItem& item) {
    using L = PairLayout;
    const int q = static_cast<int>(c.warp & 3u);  // this warp may access TMEM lanes 32q .. 32q+31
    const int h = static_cast<int>((c.warp - L::EPI_WARP0) >> 2);  // its half of the columns
    width = item.half >= 0 ? L::BLOCK_N / 4 : L::BLOCK_N / 2;
    col0 = item.n_blk * L::BLOCK_N + (item.half > 0 ? 2 * width : 0) + h * width;
    row0 = item.m_blk * L::TILE_M + static_cast<int>(c.rank) * L::CTA_M + q * 32;
    row = row0 + static_cast<int>(c.lane);
    live = row0 < p.main.rows && col0 < p.main.cols;
  }
};

__device__ __forceinline__ int sum_parts(const LossParams& p) {
  return (p.main.k_iters + kPairSumStages - 1) / kPairSumStages;
}

// Forward: a row's columns of a tile are reduced.
__global__ void __launch_bounds__(PairLayout::NUM_THREADS, 1)
    loss_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ LossParams p) {
  pair_cta<kPairRows>(maps, p, [&](const PairCta& c) {
    const int h = static_cast<int>((c.warp - PairLayout::EPI_WARP0) >> 2), parts = sum_parts(p);
    uint32_t acc = 0;
    PairItem item;
    for (int it = 0; pair_item(p, c.cluster_idx, c.num_clusters, it, item); ++it) {
      const LossPlace at(p, c, item);
      LossRow r;
      r.begin(p, at.row);  // (while the MMAs run)
      float sum[4][32];
      if (!add_parts(c, parts, at.width, at.live, acc, sum)) break;
      if (at.row0 >= p.main.rows) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = at.col0 + k * 32;
        if (k * 32 < at.width && col < p.main.cols) r.chunk(p, sum[k], at.row, col);
      }
      r.end(p, item, h, at.row);
    }
  });
}

// Gradient: a tile's logits become G. They are added in the parts of the forward pass: p = exp(z - lse) takes the difference of
// two numbers of the same size, and a row that its target dominates p - 1 behind it, so a z from one accumulator against an lse
// from parts would be most of such a row's G (the size of its logit times 2^-25 a step of 16).
__global__ void __launch_bounds__(PairLayout::NUM_THREADS, 1)
    grad_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ LossParams p) {
  using L = PairLayout;
  pair_cta<kPairRows>(maps, p, [&](const PairCta& c) {
    const int parts = sum_parts(p);
    PairStaging st{c.base + L::OFF_EPI + (c.warp - L::EPI_WARP0) * kPairStagingBytes, 0u, false};
    uint32_t acc = 0;
    PairItem item;
    for (int it = 0; pair_item(p, c.cluster_idx, c.num_clusters, it, item); ++it) {
      const LossPlace at(p, c, item);
      GradRow r;
      r.begin(p, at.row);  // (while the MMAs run)
      float sum[4][32];
      if (!add_parts(c, parts, at.width, at.live, acc, sum)) break;
      if (at.row0 >= p.main.rows) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = at.col0 + k * 32;
        if (k * 32 < at.width && col < p.main.cols) {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sum[k][j]);
          r.chunk(v, col);
          pair_store(st, c.lane, &maps.c0, v, col, at.row0, false);
        }
      }
    }
    if (c.lane == 0) bulk_wait_group<0>();
    __syncwarp();
  });
}

// ---------------------------------------------------------------- a row's parts

struct LossJoin {
  const float2* parts;  // [count][rows]
  int count, rows, vocab;
  PairProduct q;  // its tiles cut in halves have more in `extra`
  const float2* extra;
  const float* target_z;
  const long long* targets;
  float* loss;
  float* lse;
  float scale;
};

// A CTA joins 32 rows: a warp takes every 32nd part of all of them, then a row each.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) loss_join_kernel(const LossJoin p) {
  __shared__ float2 seen[kJoinWarps][33];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = log2_scale(p.scale);
  SoftmaxPart part{-INFINITY, -1.0f};
  {
    const int row = blockIdx.x * 32 + lane;
    if (row < p.rows) {
#pragma unroll 8
      for (int i = warp; i < p.count; i += kJoinWarps) {
        const float2 a = p.parts[static_cast<long long>(i) * p.rows + row];
        part = join(part, SoftmaxPart{a.x, a.y}, c);
      }
      if (p.q.split_tiles > 0) {
        constexpr int TILE_M = PairLayout::TILE_M;
        const int m_blk = row / TILE_M;
        for (int n = warp; n < p.q.num_n_blocks; n += kJoinWarps) {
          const int i = tile_index(p.q, m_blk, n) - (p.q.num_tiles - p.q.split_tiles);
          if (i < 0) continue;
          const float2* more = p.extra + 2LL * i * TILE_M + (row - m_blk * TILE_M);
          const float2 d = more[0], e = more[TILE_M];
          part = join(part, SoftmaxPart{d.x, d.y}, c);
          part = join(part, SoftmaxPart{e.x, e.y}, c);
        }
      }
    }
  }
  seen[warp][lane] = make_float2(part.m, part.others);
  __syncthreads();
  const float2 mine = seen[lane][warp];
  part = SoftmaxPart{mine.x, mine.y};
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    part = join(part, SoftmaxPart{__shfl_down_sync(0xffffffffu, part.m, o), __shfl_down_sync(0xffffffffu, part.others, o)},
                c);
  const int row = blockIdx.x * 32 + warp;
  if (lane != 0 || row >= p.rows) return;
  if (p.count == 0) part = SoftmaxPart{0.0f, static_cast<float>(p.vocab - 1)};  // K == 0: every logit is 0
  const float rest = log1pf(part.others) + (part.m - part.m);  // (an infinite maximum makes the row NaN)
  p.lse[row] = fmaf(p.scale, part.m, rest);
  if (p.loss == nullptr) return;
  const long long t = p.targets[row];
  float loss = 0.0f;
  if (t >= p.vocab) loss = __int_as_float(0x7FC00000);
  else if (t >= 0) loss = fmaf(p.scale, part.m - (p.count == 0 ? 0.0f : p.target_z[row]), rest);
  p.loss[row] = loss;
}

// ---------------------------------------------------------------- host side

enum LossKernel { kLoss = 0, kGrad = 1 };
const void* loss_kernel_of(LossKernel k) {
  return k == kLoss ? reinterpret_cast<const void*>(loss_kernel) : reinterpret_cast<const void*>(grad_kernel);
}

int loss_max_clusters(int device, LossKernel k) {
  static std::mutex mu;
  static int cache[64][2] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (device < 0 || device >= 64) return 0;
  int& n = cache[device][k];
  if (n == 0) {
    const void* kernel = loss_kernel_of(k);
    n = pair_max_clusters(&kernel, 1, false);
  }
  return n;
}

// X's rows against `cols` rows of W from its row p.first_col on, G (or nothing) to `out`.
int loss_launch(LossParams& p, LossKernel k, const void* X, long long ldx, const void* W, int K, int cols, void* out,
                long long ldo, int device, const DeviceInfo* info, cudaStream_t stream) {
  const int rows = p.main.rows;
  PairMaps m;
  int st = pair_map_in(&m.a0, X, K, rows, ldx, 128);
  if (st == GEMM_OK)
    st = pair_map_in(&m.b0, static_cast<const uint16_t*>(W) + static_cast<long long>(p.first_col) * K, K, cols, K, 64);
  m.a1 = m.c0 = m.c1 = m.c2 = m.a0;
  m.b1 = m.b2 = m.b0;
  if (out != nullptr && st == GEMM_OK) st = pair_map_out(&m.c0, out, cols, rows, ldo);
  if (st != GEMM_OK) return st;
  const int wave = loss_max_clusters(device, k);
  if (wave <= 0) return GEMM_ERR_LAUNCH;
  const int clusters = pair_schedule(&p, false, 2.0, wave, device, info);
  if (clusters < 0) return -clusters;
  void* args[] = {&m, &p};
  return pair_launch(loss_kernel_of(k), args, false, clusters, stream);
}

// Rows of 8 columns at a time, `vectors` of them to a row, into rows `ldo` apart.
__global__ void __launch_bounds__(256) copy_rows_kernel(const uint16_t* x, long long ldx, uint16_t* out, long long ldo,
                                                        int vectors, long long total) {
  pdl_launch_dependents();
  pdl_wait();
  const long long i = blockIdx.x * 256LL + threadIdx.x;
  if (i >= total) return;
  const long long row = i / vectors, v = i - row * vectors;
  *reinterpret_cast<uint4*>(out + row * ldo + 8 * v) = *reinterpret_cast<const uint4*>(x + row * ldx + 8 * v);
}

template <class... Params, class... Args>
int simple_launch(void (*kernel)(Params...), int grid, int threads, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

// A 128-byte row of a TMA box that starts off a 128-byte boundary costs a fifth sector and a second line of L2, which large
// launches feel: 1500 x 50001 x 2056 takes 221 us forward where 2048 deep takes 176. X, which every tile of columns reads
// again, is worth a copy in rows that start on the boundary where its products are large (W, as large as what is read of
// it, is not). With the copy it takes 204 forward, and 568
// instead of 596 for the gradient; 8192 x 32001 x 1000 339 and 382 without, 970 and 1022.
bool on_boundary(const void* X, long long ldx) { return (reinterpret_cast<uintptr_t>(X) & 127u) == 0 && ldx % 64 == 0; }
bool copy_pays(bool x_on_boundary, int M, int vocab, int K) {
  return !x_on_boundary && 2.0 * M * vocab * K > 1e11 && vocab > 4096;
}
long long copy_stride(int K) { return (K + 63LL) / 64 * 64; }
int copy_rows(const void* X, long long ldx, void* out, int M, int K, cudaStream_t stream) {
  const long long total = static_cast<long long>(M) * (K / 8);
  return simple_launch(copy_rows_kernel, static_cast<int>((total + 255) / 256), 256, stream,
                       static_cast<const uint16_t*>(X), ldx, static_cast<uint16_t*>(out), copy_stride(K), K / 8, total);
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

struct LossStrides {
  long long x, dx;
};
int resolve(const gemm_cross_entropy_strides_t* s, int K, LossStrides* r) {
  *r = LossStrides{K, K};
  if (s == nullptr) return GEMM_OK;
  if (s->x) r->x = s->x;
  if (s->dx) r->dx = s->dx;
  return r->x < K || r->dx < K ? GEMM_ERR_INVALID_ARG : GEMM_OK;
}

bool good_scale(float s) { return s > 0.0f && std::isfinite(s); }

size_t round_up(size_t n, size_t to) { return (n + to - 1) / to * to; }

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_cross_entropy_piece(int M, int vocab, size_t workspace) {
  if (M < 0 || vocab < 0) return -GEMM_ERR_INVALID_ARG;
  if (M == 0 || vocab == 0) return vocab;
  if (workspace == 0) workspace = kLossWorkspace;
  const size_t column = (M <= kLossRows ? 4 : 2) * static_cast<size_t>(M);  // bytes (few rows: G as two numbers)
  const long long most = std::max<long long>(
      256, static_cast<long long>(std::min<size_t>(workspace, size_t(1) << 50) / column) / 256 * 256);
  if (most >= vocab) return vocab;
  const long long pieces = (vocab + most - 1) / most;  // of about the same size
  return static_cast<int>(round_up((vocab + pieces - 1) / pieces, 256));
}

int gemm_cross_entropy_plan(int M, int vocab, int K, int wave, size_t workspace, int input_grad, int weight_grad,
                            int* products, int* copy) {
  if (M < 0 || vocab < 0 || K < 0 || wave <= 0 || products == nullptr || copy == nullptr) return GEMM_ERR_INVALID_ARG;
  const bool few = M <= kLossRows;
  PairGradient q = {};
  q.dx = input_grad ? copy : nullptr;  // (nothing is read)
  q.dw[0] = weight_grad ? copy : nullptr;
  q.rows = few ? 2 * M : M;
  q.features[0] = q.features[1] = gemm_cross_entropy_piece(M, vocab, workspace);
  q.K = K;
  q.parts = 1;
  *products = pair_gradient_is_wide(q, wave) ? 512 : 256;
  *copy = !few && copy_pays(K % 64 == 0, M, vocab, K) ? 1 : 0;
  return GEMM_OK;
}

int gemm_cross_entropy(const void* X, const void* W, const long long* targets, float* loss, float* lse, int M, int vocab,
                       int K, float scale, void* stream, const gemm_cross_entropy_strides_t* strides) {
  using L = PairLayout;
  LossStrides ld;
  if (M < 0 || vocab < 0 || K < 0 || !good_scale(scale) || resolve(strides, K, &ld) != GEMM_OK)
    return GEMM_ERR_INVALID_ARG;
  if (M == 0) return GEMM_OK;
  if (vocab == 0 || lse == nullptr || (targets == nullptr) != (loss == nullptr) ||
      (K > 0 && (X == nullptr || W == nullptr)))
    return GEMM_ERR_INVALID_ARG;
  if (K % 8 != 0 || ld.x % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if ((K > 0 && (!aligned(X, 16) || !aligned(W, 16))) || !aligned(targets, 8) || !aligned(loss, 4) || !aligned(lse, 4))
    return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  LossJoin j = {};
  j.rows = M;
  j.vocab = vocab;
  j.targets = targets;
  j.loss = loss;
  j.lse = lse;
  j.scale = scale;
  const int join_ctas = ceil_div(M, 32);
  if (K == 0) return simple_launch(loss_join_kernel, join_ctas, 32 * kJoinWarps, s, j);
  const bool few = M <= kLossRows;
  LossParams p = {};
  int st = GEMM_OK;
  size_t extra = 0;
  if (few) {
    j.count = loss_rows_ctas(vocab, info);
  } else {
    const int wave = loss_max_clusters(device, kLoss);
    if (wave <= 0) return GEMM_ERR_LAUNCH;
    st = pair_plan_product(&p.main, M, vocab, K, 128, 1, 1, L::TILE_M, L::BLOCK_N);
    if (st != GEMM_OK) return st;
    j.count = 2 * p.main.num_n_blocks;
    extra = size_t(wave) * L::TILE_M;  // (at most half a wave's tiles are cut in halves)
  }
  const size_t parts = size_t(j.count) * M;
  const bool copied = !few && copy_pays(on_boundary(X, ld.x), M, vocab, K);
  const size_t copy = copied ? size_t(M) * copy_stride(K) * 2 : 0;  // a multiple of 128
  cudaMemPool_t pool = workspace_pool(device);
  void* ws = nullptr;
  if (pool == nullptr ||
      cudaMallocFromPoolAsync(&ws, copy + (parts + extra) * sizeof(float2) + size_t(M) * 4, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  if (copy > 0) {
    st = copy_rows(X, ld.x, ws, M, K, s);
    X = ws;
    ld.x = copy_stride(K);
  }
  float2* const seen = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + copy);
  float* const target_z = reinterpret_cast<float*>(seen + parts + extra);
  if (st != GEMM_OK) {
    // (nothing to launch)
  } else if (few) {
    st = run_loss_rows(LossRowsOperands{X, W, targets, seen, target_z, ld.x, M, vocab, K, scale}, device, info, s);
  } else {
    p.scale = scale;
    p.targets = targets;
    p.vocab = vocab;
    p.parts = seen;
    p.extra = seen + parts;
    p.target_z = target_z;
    st = loss_launch(p, kLoss, X, ld.x, W, K, vocab, nullptr, 0, device, info, s);
    j.q = p.main;
    j.extra = p.extra;
  }
  if (st == GEMM_OK) {
    j.parts = seen;
    j.target_z = target_z;
    st = simple_launch(loss_join_kernel, join_ctas, 32 * kJoinWarps, s, j);
  }
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

int gemm_cross_entropy_backward(const void* X, const void* W, const long long* targets, const float* lse,
                                const float* dloss, const float* dlse, void* dX, void* dW, int M, int vocab, int K,
                                float scale, size_t workspace, void* stream,
                                const gemm_cross_entropy_strides_t* strides) {
  using L = PairLayout;
  LossStrides ld;
  if (M < 0 || vocab < 0 || K < 0 || !good_scale(scale) || resolve(strides, K, &ld) != GEMM_OK)
    return GEMM_ERR_INVALID_ARG;
  if (vocab == 0 && M > 0) return GEMM_ERR_INVALID_ARG;
  if ((targets == nullptr) != (dloss == nullptr)) return GEMM_ERR_INVALID_ARG;
  if ((dX == nullptr && dW == nullptr) || K == 0 || vocab == 0) return GEMM_OK;
  if (M > 0 && (X == nullptr || W == nullptr || lse == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (K % 8 != 0 || ld.x % 8 != 0 || ld.dx % 8 != 0) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(X, 16) || !aligned(W, 16) || !aligned(dX, 16) || !aligned(dW, 16) || !aligned(targets, 8) ||
      !aligned(lse, 4) || !aligned(dloss, 4) || !aligned(dlse, 4))
    return GEMM_ERR_MISALIGNED;
  if (M == 0 && dW == nullptr) return GEMM_OK;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {  // a sum over no rows
    if (cudaMemsetAsync(dW, 0, size_t(vocab) * K * 2, s) == cudaSuccess) return GEMM_OK;
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  const int piece = gemm_cross_entropy_piece(M, vocab, workspace);
  const bool pieces = piece < vocab;
  const long long ldg = static_cast<long long>(round_up(piece, 64));  // (rows on 128-byte boundaries, see copy_rows)
  const bool few = M <= kLossRows;
  const int g_rows = few ? 2 * M : M;  // (see cross_entropy_rows.cu)
  PairGradient q = {};
  q.x = X;
  q.ldg = ldg;
  q.ldx = ld.x;
  q.lddx = ld.dx;
  q.rows = g_rows;
  q.K = K;
  q.parts = 1;
  q.even = true;
  q.keep_sums = (pieces || few) && dX != nullptr;
  auto at = [&](const void* p, int row) {
    return static_cast<void*>(const_cast<uint16_t*>(static_cast<const uint16_t*>(p)) + static_cast<long long>(row) * K);
  };
  auto select = [&](int first) {  // the piece from column `first` on
    q.features[0] = q.features[1] = std::min(piece, vocab - first);
    q.w[0] = at(W, first);
    q.dx = dX;
    q.dw[0] = dW != nullptr ? at(dW, first) : nullptr;
    q.add = first > 0;
  };
  select(0);
  PairGradientPlan plan;
  int st = pair_gradient_plan(q, device, &plan);
  if (st != GEMM_OK) return st;
  const size_t g_bytes = round_up(size_t(g_rows) * ldg * 2, 256);
  const bool copied = few ? dW != nullptr : copy_pays(on_boundary(X, ld.x), M, vocab, K);
  const size_t copy = copied ? round_up(size_t(g_rows) * copy_stride(K) * 2, 256) : 0;
  cudaMemPool_t pool = workspace_pool(device);
  void* ws = nullptr;
  if (pool == nullptr || cudaMallocFromPoolAsync(&ws, g_bytes + copy + plan.sums * 4, pool, s) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_OUT_OF_MEMORY;
  }
  if (copy > 0) {
    void* const to = static_cast<uint8_t*>(ws) + g_bytes;
    if (!few) {
      st = copy_rows(X, ld.x, to, M, K, s);
      X = to;
      ld.x = copy_stride(K);
    }
    q.x = to;
    q.ldx = copy_stride(K);
  }
  float* const sums = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + g_bytes + copy);
  q.g[0] = ws;
  const int slices = q.most_slices = plan.p.main.slices;
  const bool join = plan.sums > 0;
  for (int first = 0; first < vocab && st == GEMM_OK; first += q.features[0]) {  // (no sum of them passes 31 bits)
    select(first);
    LossParams p = {};
    p.scale = scale;
    p.first_col = first;
    p.grad = LossGradient{targets, lse, dloss, dlse, M, vocab, first, scale};
    if (few) {
      uint16_t* const twice = copied ? static_cast<uint16_t*>(const_cast<void*>(q.x)) : nullptr;
      st = run_loss_rows_gradient(LossRowsOperands{X, q.w[0], nullptr, nullptr, nullptr, ld.x, M, q.features[0], K, scale},
                                  LossRowsGradient{p.grad, static_cast<uint16_t*>(ws), ldg, twice, q.ldx}, device, info, s);
    } else {
      st = pair_plan_product(&p.main, M, q.features[0], K, 128, 1, 1, L::TILE_M, L::BLOCK_N);
      if (st == GEMM_OK) st = loss_launch(p, kGrad, X, ld.x, W, K, q.features[0], ws, ldg, device, info, s);
    }
    // (a last piece of fewer slices adds to the first ones)
    if (st == GEMM_OK && first > 0) st = pair_gradient_plan(q, device, &plan);
    if (st == GEMM_OK) st = pair_gradient_launch(q, &plan, sums, device, info, s);
  }
  if (st == GEMM_OK && join) st = pair_gradient_join(sums, slices, dX, ld.dx, M, K, s, few);
  if (cudaFreeAsync(ws, s) != cudaSuccess && st == GEMM_OK) st = GEMM_ERR_LAUNCH;
  return st;
}

}  // extern "C"
