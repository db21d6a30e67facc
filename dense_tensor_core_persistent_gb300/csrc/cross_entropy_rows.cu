// cross_entropy_rows.cu -- the logits of the head's cross entropy for up to 64 rows, from a single position on: their
// softmax statistics, or what they become in the gradient.
//
// W's bytes are the bound, and on the 256-row pair tile most of each MMA would multiply rows that X does not have. Here 128
// rows of W are the MMA's M and the rows of X its N: accumulator lane v holds the logits of token v, columns are the rows
// of X. A CTA takes a run of the vocabulary in boxes of 32 tokens, so all CTAs stream the same bytes whatever the
// vocabulary; its tiles are of up to four boxes and about the same size (a last one of what is left, which has less on its
// way at a time, cost 30 x 100000 x 2048 72 us instead of 69). The depth is summed in parts of 128 (pair_tile.cuh says why),
// which the epilogue adds in FP32: a loss of a few rows has no others to average its error with, and here short parts cost
// nothing. 4 x 9713 x 1008, mean over 24 inputs against 64 bits: lse 7.5e-8 and loss 1.3e-7 of their size, with parts of 512
// 3.0e-7 and 5.5e-7 (FP32 products 3.4e-8 and 1.6e-7); parts of 64 would be 5.1e-8 and 1.1e-7 at 1.4 times the time.
// The softmax is one pass: a thread keeps, for its lane's tokens and each of its rows of X, the maximum and the sum of the
// others relative to it through all of the CTA's tiles; lanes, warps and (in the joining kernel) CTAs are joined at the
// end, in a fixed order.
//
// Measured on GB300 with W of 131072 x 4096 (1.07 GB, 158 us at the rate of a copy): 1 row 158 to 163 us, where the pair
// tile took 290; 64 rows 160 to 166, where the pair tile's 65 rows take 193 and its 128 191.
//
// In the gradient G's two products have room for more rows than X has: their tiles are 256 rows, their stages 128. So G is
// kept as two BF16 numbers, the second what the first one's rounding left, as rows of their own, and X's rows twice for the
// product with both; the error of dX and dW against 64 bits is that of their own rounding (4 x 9713 x 1008 1.66e-3, with one
// number 2.3e-3 in the mean and 3.0e-3 at the most). It costs 64 x 131072 x 4096 569 -> 579 us, 64 x 16000 x 1024 29 -> 32.
//
// One persistent CTA per SM. Warp roles: 0 loads W, 2 loads X, 1 allocates TMEM and issues the MMAs, 3 copies X for the
// gradient, 4..11 epilogue, two to each TMEM lane quadrant with half of X's rows each. Two accumulators in TMEM.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "loss_common.cuh"

namespace dtcp {
namespace {

struct LossRowsParams {
  LossRowsOperands x;
  LossRowsGradient grad;
  int k_iters, boxes;  // stages of a tile; boxes of 32 tokens in all
  int n;               // the MMA's N: the rows of X, rounded up to a multiple of 16
  unsigned* status;
  unsigned long long wait_limit_ns;
};

template <int X_ROWS>
struct LossRowsLayout {
  static constexpr int BOX = 32, TILE_BOXES = 4;
  // 128-byte swizzle rows of K per stage; MMAs; elements, which are a part of the depth with an accumulator of its own
  static constexpr int ATOMS = 2, KSTEPS = 8, STAGE_K = 128;
  static constexpr int BOX_BYTES = BOX * 128;
  static constexpr int W_ATOM_BYTES = TILE_BOXES * BOX_BYTES, X_ATOM_BYTES = X_ROWS * 128;
  static constexpr int W_BYTES = ATOMS * W_ATOM_BYTES, X_BYTES = ATOMS * X_ATOM_BYTES;
  static constexpr int STAGES = X_ROWS == 16 ? 6 : 4;
  static constexpr int TMEM_COLS = 2 * X_ROWS;
  static constexpr int WARP_W = 0, WARP_MMA = 1, WARP_X = 2, WARP_COPY = 3, EPI_WARP0 = 4, EPI_WARPS = 8;
  static constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
  static constexpr int COLS = X_ROWS / 2;  // rows of X of an epilogue warp
  static constexpr int OFF_W = 0;
  static constexpr int OFF_X = STAGES * W_BYTES;
  static constexpr int OFF_JOIN = OFF_X + STAGES * X_BYTES;       // [4][X_ROWS] (m, others)
  static constexpr int OFF_ROWS = OFF_JOIN + 4 * X_ROWS * 8;      // [EPI_WARPS][COLS]: forward targets, else float4
  static constexpr int OFF_BAR = OFF_ROWS + EPI_WARPS * COLS * 16;
  // full[S], empty[S], tmem_full[2], tmem_empty[2], drain
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 4 + 1024;  // slack to align the base to 1024 bytes
  static_assert(SMEM_BYTES <= 232448, "exceeds 227 KB of shared memory per CTA");
};

// Joins the warp's lanes for each of COLS columns: lanes exchange halves of their columns until each has one, 31 joins a
// lane for 32 columns where column by column would be 160 (64 x 131072 x 1024 54.4 us by columns, 47.7 so). Lane l has
// column l * COLS / 32.
template <int COLS>
__device__ __forceinline__ SoftmaxPart join_lanes(SoftmaxPart (&s)[COLS], float c) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16, n = COLS / 2; o > 0; o >>= 1, n >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int j = 0; j < (n > 0 ? n : 1); ++j) {
      const SoftmaxPart keep = n > 0 && up ? s[j + n] : s[j], give = n > 0 && !up ? s[j + n] : s[j];
      s[j] = join(keep, SoftmaxPart{__shfl_xor_sync(0xffffffffu, give.m, o), __shfl_xor_sync(0xffffffffu, give.others, o)}, c);
    }
  }
  return s[0];
}

// COLS columns of this warp's TMEM lanes.
template <int COLS>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&v)[COLS]) {
  static_assert(COLS == 8 || COLS == 32, "columns of an epilogue warp");
  if constexpr (COLS == 8) tmem_ld_32x32b_x8(taddr, v);
  else tmem_ld_32x32b_x32(taddr, v);
}

template <int X_ROWS, bool GRAD>
__global__ void __launch_bounds__(LossRowsLayout<X_ROWS>::NUM_THREADS, 1)
    loss_rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ LossRowsParams p) {
  using L = LossRowsLayout<X_ROWS>;
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
  pdl_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  // this CTA's boxes
  const int box0 = static_cast<int>(static_cast<long long>(blockIdx.x) * p.boxes / gridDim.x);
  const int box1 = static_cast<int>((static_cast<long long>(blockIdx.x) + 1) * p.boxes / gridDim.x);
  const int tiles = (box1 - box0 + L::TILE_BOXES - 1) / L::TILE_BOXES;  // of about the same size
  const int each = (box1 - box0) / tiles, one_more = (box1 - box0) % tiles;
  auto tile_box = [&](int t) { return box0 + t * each + min(t, one_more); };

  if ((warp == L::WARP_W || warp == L::WARP_X) && lane == 0) {
    // ------------------------------------------------------------ producers
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    for (int t = 0; t < tiles && ok; ++t) {
      const int b = tile_box(t), boxes = tile_box(t + 1) - b;
      for (int k = 0; k < p.k_iters; ++k) {
        if (!wait_phase_inline(bar_empty + 8 * stage, phase ^ 1u, wctx, status_code(kRoleProducer, stage))) {
          ok = false;
          break;
        }
        const uint32_t full = bar_full + 8 * stage;
        if (warp == L::WARP_W) {
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(L::ATOMS * boxes * L::BOX_BYTES));
#pragma unroll
          for (int a = 0; a < L::ATOMS; ++a) {
            const uint32_t dst = base + L::OFF_W + stage * L::W_BYTES + a * L::W_ATOM_BYTES;
            for (int c = 0; c < boxes; ++c)
              tma_load_2d(dst + c * L::BOX_BYTES, &map_w, k * L::STAGE_K + a * 64, (b + c) * L::BOX, full);
          }
        } else {
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(L::ATOMS * p.n * 128));
#pragma unroll
          for (int a = 0; a < L::ATOMS; ++a)
            tma_load_2d(base + L::OFF_X + stage * L::X_BYTES + a * L::X_ATOM_BYTES, &map_x, k * L::STAGE_K + a * 64, 0,
                        full);
        }
        stage = stage + 1 == L::STAGES ? 0u : stage + 1;
        phase = stage == 0 ? phase ^ 1u : phase;
      }
    }
    if (!ok) settle_after_abort();
  } else if (warp == L::WARP_MMA && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16(128, p.n);
    const uint64_t a0 = umma_desc_sw128(base + L::OFF_W), b0 = umma_desc_sw128(base + L::OFF_X);
    uint32_t stage = 0, phase = 0, acc = 0;
    bool ok = true;
    for (int t = 0; t < tiles && ok; ++t) {
      for (int k = 0; k < p.k_iters; ++k, ++acc) {
        const uint32_t slot = acc & 1u;
        if (!wait_phase_inline(bar_tempty + 8 * slot, ((acc >> 1) & 1u) ^ 1u, wctx, status_code(kRoleMma, 0x100 + slot))) {
          ok = false;
          break;
        }
        if (!wait_phase_inline(bar_full + 8 * stage, phase, wctx, status_code(kRoleMma, stage))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d = tmem_base + slot * X_ROWS;
        const uint64_t a = umma_desc_advance(a0, stage * L::W_BYTES), b = umma_desc_advance(b0, stage * L::X_BYTES);
        const int left = p.x.depth - k * L::STAGE_K;  // a ragged last stage: only the MMAs that hold any of it
        const int steps = left >= L::STAGE_K ? L::KSTEPS : (left + 15) / 16;
        auto one = [&](int kk) {
          const uint32_t in_atom = static_cast<uint32_t>(kk % 4) * 32u, atom = static_cast<uint32_t>(kk / 4);
          mma_f16<1>(d, umma_desc_advance(a, atom * L::W_ATOM_BYTES + in_atom),
                     umma_desc_advance(b, atom * L::X_ATOM_BYTES + in_atom), idesc, kk != 0 ? 1u : 0u);
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
        mma_commit_local(bar_tfull + 8 * slot);
      }
    }
    if (!ok) {
      // let issued MMAs finish before TMEM is released (bounded: they finish or the limit passes)
      mma_commit_local(bar_drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait_suspend(bar_drain, 0, 20000u) && globaltimer_ns() - t0 < wctx.limit_ns) {
      }
      settle_after_abort();
    }
  }
  if constexpr (GRAD) {
    if (warp == L::WARP_COPY && p.grad.x_twice != nullptr) {  // X's rows twice, 8 columns at a time
      const long long vectors = p.x.depth / 8, all = p.x.rows * vectors;
      for (long long i = blockIdx.x * 32u + lane; i < all; i += gridDim.x * 32u) {
        const long long row = i / vectors, col = (i - row * vectors) * 8;
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x.x) + row * p.x.ldx + col);
        uint16_t* const to = p.grad.x_twice + row * p.grad.ldx_twice + col;
        *reinterpret_cast<uint4*>(to) = v;
        *reinterpret_cast<uint4*>(to + p.x.rows * p.grad.ldx_twice) = v;
      }
    }
  }
  float2* const joined = reinterpret_cast<float2*>(smem + L::OFF_JOIN);
  const float c = log2_scale(p.x.scale);
  if (warp >= L::EPI_WARP0) {
    // ------------------------------------------------------------ epilogue
    const uint32_t q = warp & 3u;                                    // TMEM lanes 32q .. 32q+31
    const int col0 = static_cast<int>((warp - L::EPI_WARP0) >> 2) * L::COLS;  // its rows of X
    const bool live = col0 < p.x.rows;
    // of its rows: the target's token (no target, and one past the vocabulary: none); in the gradient its factors too
    uint8_t* const of_rows = smem + L::OFF_ROWS + (warp - L::EPI_WARP0) * L::COLS * 16;
    int* const target = reinterpret_cast<int*>(of_rows);
    float4* const factors = reinterpret_cast<float4*>(of_rows);
    uint32_t dead = 0;
    if constexpr (GRAD) {
      const GradientRow g(p.grad.row, col0 + static_cast<int>(lane));
      if (lane < L::COLS) {
        const int token = g.target >= 0 && g.target < p.x.vocab ? static_cast<int>(g.target) : -1;
        factors[lane] = make_float4(g.lse, g.softmax, g.onehot, __int_as_float(token));
      }
      dead = __ballot_sync(0xffffffffu, g.dead);
    } else if (lane < L::COLS) {
      const int r = col0 + static_cast<int>(lane);
      const long long t = p.x.targets != nullptr && r < p.x.rows ? p.x.targets[r] : -1;
      target[lane] = t >= 0 && t < p.x.vocab ? static_cast<int>(t) : -1;
    }
    __syncwarp();
    SoftmaxPart s[L::COLS];
#pragma unroll
    for (int j = 0; j < L::COLS; ++j) s[j] = SoftmaxPart{-INFINITY, -1.0f};
    uint32_t acc = 0;
    bool ok = true;
    for (int t = 0; t < tiles && ok; ++t) {
      const int b = tile_box(t), token = (b + static_cast<int>(q)) * L::BOX + static_cast<int>(lane);
      const bool in = b + static_cast<int>(q) < tile_box(t + 1) && token < p.x.vocab;
      float z[L::COLS];
#pragma unroll 1
      for (int part = 0; part < p.k_iters; ++part, ++acc) {
        const uint32_t slot = acc & 1u;
        if (!wait_phase_warp(bar_tfull + 8 * slot, (acc >> 1) & 1u, wctx, status_code(kRoleEpilogue, slot))) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        uint32_t v[L::COLS];
        tmem_ld_cols<L::COLS>(tmem_base + ((q * 32u) << 16) + slot * X_ROWS + static_cast<uint32_t>(col0), v);
        tmem_ld_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(bar_tempty + 8 * slot);
#pragma unroll
        for (int j = 0; j < L::COLS; ++j) z[j] = part == 0 ? __uint_as_float(v[j]) : z[j] + __uint_as_float(v[j]);
      }
      if (!ok || !live || !in) continue;
      if constexpr (GRAD) {
        uint16_t* const to = p.grad.g + col0 * p.grad.ldg + token;
        const long long half = p.x.rows * p.grad.ldg;
#pragma unroll
        for (int j = 0; j < L::COLS; ++j) {
          if (col0 + j >= p.x.rows) break;
          const float4 f = factors[j];
          float v = gradient_of(z[j], p.x.scale, f.x, f.y, (dead >> j & 1u) != 0u);
          if (__float_as_int(f.w) == token) v -= f.z;
          const uint32_t high = pack_bf16x2_rn(__float_as_uint(v), 0u) & 0xFFFFu;
          const float left = v - __uint_as_float(high << 16);  // (of an infinity NaN, as of a NaN)
          to[j * p.grad.ldg] = static_cast<uint16_t>(high);
          to[j * p.grad.ldg + half] = static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(left), 0u) & 0xFFFFu);
        }
      } else {
#pragma unroll
        for (int j = 0; j < L::COLS; ++j) {
          if (target[j] == token) p.x.target_z[col0 + j] = z[j];
          // the new logit is the maximum, or one of the others; minus infinity adds nothing to either
          const float d = z[j] - s[j].m, e = ex2_approx(-fabsf(d) * c);
          if (z[j] != -INFINITY) s[j].others = d > 0.0f ? (s[j].others + 1.0f) * e : s[j].others + e;
          s[j].m = fmaxf(s[j].m, z[j]);
        }
      }
    }
    if constexpr (!GRAD) {
      const SoftmaxPart all = join_lanes<L::COLS>(s, c);
      if (lane % (32 / L::COLS) == 0) joined[q * X_ROWS + col0 + lane / (32 / L::COLS)] = make_float2(all.m, all.others);
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (!GRAD && threadIdx.x < static_cast<unsigned>(p.x.rows)) {
    SoftmaxPart s{-INFINITY, -1.0f};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = joined[q * X_ROWS + threadIdx.x];
      s = join(s, SoftmaxPart{v.x, v.y}, c);
    }
    p.x.parts[static_cast<long long>(blockIdx.x) * p.x.rows + threadIdx.x] = make_float2(s.m, s.others);
  }
  if (warp == L::WARP_MMA) {
    tc_fence_after_sync();
    tmem_dealloc<1>(tmem_base, L::TMEM_COLS);
  }
}

template <int X_ROWS, bool GRAD>
int launch_rows(const LossRowsOperands& x, const LossRowsGradient& grad, int device, const DeviceInfo* info,
                cudaStream_t stream) {
  using L = LossRowsLayout<X_ROWS>;
  const auto kernel = loss_rows_kernel<X_ROWS, GRAD>;
  {
    static std::mutex mu;
    static bool done[64] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!done[device & 63]) {
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_BYTES) != cudaSuccess) {
        cudaGetLastError();
        return GEMM_ERR_LAUNCH;
      }
      done[device & 63] = true;
    }
  }
  LossRowsParams p;
  p.x = x;
  p.grad = grad;
  p.n = ceil_div(x.rows, 16) * 16;
  p.k_iters = ceil_div(x.depth, L::STAGE_K);
  p.boxes = ceil_div(x.vocab, L::BOX);
  p.status = device_status_word(device);
  p.wait_limit_ns = RunOptions().wait_limit_ns;
  if (p.status == nullptr) return GEMM_ERR_NO_DEVICE;
  CUtensorMap w, rows;
  int st = encode_tmap_2d(&w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x.w, x.depth, x.vocab, uint64_t(x.depth) * 2, 64, L::BOX,
                          CU_TENSOR_MAP_SWIZZLE_128B);
  if (st == GEMM_OK)
    st = encode_tmap_2d(&rows, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x.x, x.depth, x.rows, uint64_t(x.ldx) * 2, 64, p.n,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != GEMM_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(loss_rows_ctas(x.vocab, info)), 1, 1);
  cfg.blockDim = dim3(L::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = L::SMEM_BYTES;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, w, rows, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

}  // namespace

int loss_rows_ctas(int vocab, const DeviceInfo* info) { return std::min(ceil_div(vocab, 32), info->num_sms); }

int run_loss_rows(const LossRowsOperands& p, int device, const DeviceInfo* info, cudaStream_t stream) {
  return p.rows <= 16 ? launch_rows<16, false>(p, LossRowsGradient{}, device, info, stream)
                      : launch_rows<64, false>(p, LossRowsGradient{}, device, info, stream);
}

int run_loss_rows_gradient(const LossRowsOperands& p, const LossRowsGradient& grad, int device, const DeviceInfo* info,
                           cudaStream_t stream) {
  return p.rows <= 16 ? launch_rows<16, true>(p, grad, device, info, stream)
                      : launch_rows<64, true>(p, grad, device, info, stream);
}

}  // namespace dtcp
