// glu_few.cu -- the gated feed-forward block for few rows (decoding steps): H = act(X Wg^T) * (X Wu^T)
// with at most 16 rows of X, BF16 or E4M3 operands, FP32 accumulation.
//
// Every byte of Wg and Wu is used for at most 16 rows, so the bytes of the weights are the bound and
// the matrix instructions only have to keep out of the loads' way. The weights go from global memory
// straight into mma.sync fragments, without shared memory or barriers: a warp's A tile is 16 features,
// its B tile 8 rows of X. The sum's order along K is free, so lane t of a row's four lanes takes 16
// contiguous bytes (8 BF16 or 16 E4M3) and feeds 8 of them to each of two MMAs, X's lanes alike.
// A CTA computes 16 features of g and of u; its warps take interleaved blocks of K, and their partial
// sums meet in shared memory in a fixed order, where the activation and the product are applied.
// N / 16 CTAs of 4 warps fill the SMs several times over, so that the last wave costs little.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "glu_act.cuh"
#include "host_common.h"

namespace dtcp {
namespace {

constexpr int kFewWarps = 4;
constexpr int kFewFeatures = 16;  // per CTA, of each of g and u

// Weights are read once: not kept in L1.
__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// d += A (16 features x 32 bytes of K) * B (8 rows x 32 bytes of K).
template <bool E4M3>
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (E4M3)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr int kBlockBytes = 128;               // of K, per row and step: two chunks of 16 bytes per lane
constexpr int kChunks = kBlockBytes / 64;

template <int NT>
struct FewBlock {
  uint4 g[2][kChunks], u[2][kChunks];  // features lane / 4 and lane / 4 + 8
  uint4 x[NT][kChunks];                // rows 8 n + lane / 4
};

template <bool E4M3, int NT>
__global__ void __launch_bounds__(32 * kFewWarps) glu_few_kernel(const GluFewParams p) {
  __shared__ float part[kFewWarps][2][NT * 8][kFewFeatures];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = lane >> 2, t = lane & 3;
  constexpr int SIZE = E4M3 ? 1 : 2;
  const long long row_bytes = static_cast<long long>(p.depth) * SIZE;
  const int f0 = blockIdx.x * kFewFeatures;
  pdl_launch_dependents();
  pdl_wait();
  const uint8_t* wg[2];
  const uint8_t* wu[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // features past the last one repeat it; they are not stored
    const long long f = min(f0 + grp + 8 * i, p.features - 1);
    wg[i] = static_cast<const uint8_t*>(p.wg) + f * row_bytes;
    wu[i] = static_cast<const uint8_t*>(p.wu) + f * row_bytes;
  }
  const uint8_t* x[NT];
  bool live[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    live[n] = 8 * n + grp < p.rows;
    x[n] = static_cast<const uint8_t*>(p.x) + (live[n] ? 8 * n + grp : 0) * p.ldx * SIZE;
  }
  float ag[NT][4], au[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) ag[n][j] = au[n][j] = 0.0f;

  auto load = [&](FewBlock<NT>& b, long long k) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const long long at = k + c * 64 + t * 16;
      const bool in = at < row_bytes;  // K is a whole number of 16-byte chunks
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b.g[i][c] = in ? load_stream(wg[i] + at) : make_uint4(0u, 0u, 0u, 0u);
        b.u[i][c] = in ? load_stream(wu[i] + at) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        b.x[n][c] = in && live[n] ? *reinterpret_cast<const uint4*>(x[n] + at) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto multiply = [&](const FewBlock<NT>& b) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16x8<E4M3>(ag[n], b.g[0][c].x, b.g[1][c].x, b.g[0][c].y, b.g[1][c].y, b.x[n][c].x, b.x[n][c].y);
        mma_16x8<E4M3>(au[n], b.u[0][c].x, b.u[1][c].x, b.u[0][c].y, b.u[1][c].y, b.x[n][c].x, b.x[n][c].y);
        mma_16x8<E4M3>(ag[n], b.g[0][c].z, b.g[1][c].z, b.g[0][c].w, b.g[1][c].w, b.x[n][c].z, b.x[n][c].w);
        mma_16x8<E4M3>(au[n], b.u[0][c].z, b.u[1][c].z, b.u[0][c].w, b.u[1][c].w, b.x[n][c].z, b.x[n][c].w);
      }
  };
  // two blocks in registers: one in flight while the other is multiplied
  constexpr long long STEP = static_cast<long long>(kFewWarps) * kBlockBytes;
  FewBlock<NT> even, odd;
  load(even, warp * kBlockBytes);
  for (long long k = warp * kBlockBytes; k < row_bytes; k += 2 * STEP) {
    load(odd, k + STEP);
    multiply(even);
    load(even, k + 2 * STEP);
    multiply(odd);
  }
  // lane's accumulators: features grp and grp + 8, rows 2t and 2t + 1 of each eight
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      part[warp][0][8 * n + 2 * t + (j & 1)][grp + 8 * (j >> 1)] = ag[n][j];
      part[warp][1][8 * n + 2 * t + (j & 1)][grp + 8 * (j >> 1)] = au[n][j];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < p.rows * kFewFeatures; i += 32 * kFewWarps) {
    const int f = i % kFewFeatures, row = i / kFewFeatures;
    if (f0 + f >= p.features) continue;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      g += part[w][0][row][f];
      u += part[w][1][row][f];
    }
    if constexpr (E4M3) {
      g *= p.x_scale[row] * p.g_scale[f0 + f];
      u *= p.x_scale[row] * p.u_scale[f0 + f];
    }
    const float h = glu_act(g, p.act) * u;
    p.h[row * p.ldh + f0 + f] = static_cast<uint16_t>(pack_bf16x2_rn(__float_as_uint(h), 0u) & 0xFFFFu);
    if (p.preact != nullptr) {
      float* pre = p.preact + static_cast<long long>(row) * 2 * p.features + f0 + f;
      pre[0] = g;
      pre[p.features] = u;
    }
  }
}

}  // namespace

int run_glu_few(const GluFewParams& p, bool e4m3, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(p.features, kFewFeatures)), 1, 1);
  cfg.blockDim = dim3(32 * kFewWarps, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = e4m3 ? (p.rows <= 8 ? glu_few_kernel<true, 1> : glu_few_kernel<true, 2>)
                           : (p.rows <= 8 ? glu_few_kernel<false, 1> : glu_few_kernel<false, 2>);
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

}  // namespace dtcp
