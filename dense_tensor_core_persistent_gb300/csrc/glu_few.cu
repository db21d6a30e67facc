// glu_few.cu -- the gated feed-forward block for few rows (decoding steps): H = act(X Wg^T) * (X Wu^T)
// with at most 8 rows of X, BF16 or E4M3 operands, FP32 accumulation.
//
// Every byte of Wg and Wu is used for at most 8 rows, so the bytes of the weights are the bound and
// the matrix instructions only have to keep out of the loads' way. The weights go from global memory
// straight into mma.sync fragments, without shared memory or barriers: a warp's A tile is 16 features,
// its B tile 8 rows of X. The sum's order along K is free, so lane t of a row's four lanes takes 16
// contiguous bytes of it, and X's lanes alike; E4M3 values become FP16 ones (exactly) on the way.
// A CTA computes 16 features of g and of u; its warps take interleaved blocks of K, and their partial
// sums meet in shared memory in a fixed order, where the activation and the product are applied.
// N / 16 CTAs of 4 warps fill the SMs several times over, so that the last wave costs little.
// Measured on GB300, 1 row x 28672 x 8192: BF16 141 us (6.7 TB/s of weights), E4M3 74 us (6.3).
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

// Two E4M3 values (first in the low byte) as two FP16 ones.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
  return r;
}

// d += A (16 features x 16 of K) * B (8 rows x 16 of K), BF16 or FP16.
template <bool FP16>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  if constexpr (FP16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
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

__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// g and u += the products of one chunk of 16 bytes of K per lane: features lane / 4 and lane / 4 + 8, a row of X.
template <bool E4M3>
__device__ __forceinline__ void multiply_chunk(float (&ag)[4], float (&au)[4], const uint4& g0, const uint4& g1,
                                               const uint4& u0, const uint4& u1, const uint4& x) {
  if constexpr (E4M3) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // four values of K per word: one MMA
      const uint32_t x0 = e4m3x2_f16x2(word(x, i)), x1 = e4m3x2_f16x2(word(x, i) >> 16);
      mma_16x8x16<true>(ag, e4m3x2_f16x2(word(g0, i)), e4m3x2_f16x2(word(g1, i)), e4m3x2_f16x2(word(g0, i) >> 16),
                        e4m3x2_f16x2(word(g1, i) >> 16), x0, x1);
      mma_16x8x16<true>(au, e4m3x2_f16x2(word(u0, i)), e4m3x2_f16x2(word(u1, i)), e4m3x2_f16x2(word(u0, i) >> 16),
                        e4m3x2_f16x2(word(u1, i) >> 16), x0, x1);
    }
  } else {
    mma_16x8x16<false>(ag, g0.x, g1.x, g0.y, g1.y, x.x, x.y);
    mma_16x8x16<false>(au, u0.x, u1.x, u0.y, u1.y, x.x, x.y);
    mma_16x8x16<false>(ag, g0.z, g1.z, g0.w, g1.w, x.z, x.w);
    mma_16x8x16<false>(au, u0.z, u1.z, u0.w, u1.w, x.z, x.w);
  }
}

constexpr int kBlockBytes = 128;               // of K, per row and step: two chunks of 16 bytes per lane
constexpr int kChunks = kBlockBytes / 64;

struct FewBlock {
  uint4 g[2][kChunks], u[2][kChunks];  // features lane / 4 and lane / 4 + 8
  uint4 x[kChunks];                    // row lane / 4
};

template <bool E4M3>
__global__ void __launch_bounds__(32 * kFewWarps) glu_few_kernel(const GluFewParams p) {
  __shared__ float part[kFewWarps][2][kGluFewRows][kFewFeatures];
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
  const bool live = grp < p.rows;
  const uint8_t* x = static_cast<const uint8_t*>(p.x) + (live ? grp : 0) * p.ldx * SIZE;
  float ag[4] = {0.0f, 0.0f, 0.0f, 0.0f}, au[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  auto load = [&](FewBlock& b, long long k) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const long long at = k + c * 64 + t * 16;
      const bool in = at < row_bytes;  // K is a whole number of 16-byte chunks
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b.g[i][c] = in ? load_stream(wg[i] + at) : make_uint4(0u, 0u, 0u, 0u);
        b.u[i][c] = in ? load_stream(wu[i] + at) : make_uint4(0u, 0u, 0u, 0u);
      }
      b.x[c] = in && live ? *reinterpret_cast<const uint4*>(x + at) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  auto multiply = [&](const FewBlock& b) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      multiply_chunk<E4M3>(ag, au, b.g[0][c], b.g[1][c], b.u[0][c], b.u[1][c], b.x[c]);
  };
  // two blocks in registers: one in flight while the other is multiplied
  constexpr long long STEP = static_cast<long long>(kFewWarps) * kBlockBytes;
  FewBlock even, odd;
  load(even, warp * kBlockBytes);
  for (long long k = warp * kBlockBytes; k < row_bytes; k += 2 * STEP) {
    load(odd, k + STEP);
    multiply(even);
    load(even, k + 2 * STEP);
    multiply(odd);
  }
  // lane's accumulators: features grp and grp + 8, rows 2t and 2t + 1
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    part[warp][0][2 * t + (j & 1)][grp + 8 * (j >> 1)] = ag[j];
    part[warp][1][2 * t + (j & 1)][grp + 8 * (j >> 1)] = au[j];
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
  const auto kernel = e4m3 ? glu_few_kernel<true> : glu_few_kernel<false>;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

}  // namespace dtcp
