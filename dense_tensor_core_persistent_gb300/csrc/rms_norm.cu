// rms_norm.cu -- root-mean-square norm of the rows of a residual stream, with the residual's
// addition in front and the operand of the next product behind: BF16, E4M3 with one scale a
// row, or NVFP4 (E2M1 codes, one E4M3 scale per 16) as gemm_nvfp4 reads it; and its gradient.
//
//   s = bf16(x + r),  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * w
//   xh = s * rstd,  c = mean(dy * w * xh),  dx = rstd * (dy * w - xh * c) + ds,
//   dw = sum over rows of dy * xh
//
// The norm reads the rounded stream s, the one that later layers and the gradient see.
// All sums are FP32; every output is rounded once from FP32.
//
// Both directions are bound by the bytes they move (forward at most 8 per element, backward 8),
// so a row is read once: a CTA keeps the whole row in registers between its reduction and its
// output (groups of 8 columns per thread, up to 4 groups x 1024 threads = 32768 columns).
// CTAs are persistent and step over rows by the grid size, so a thread always owns the same
// columns: the weight is read once per CTA and the weight's gradient is summed in registers,
// one partial row per CTA, which a second kernel adds in a fixed order (no atomics).
//
// Rows that no 16-byte vector divides: the groups of a row start at its 16-byte boundary, so
// all but the first and last of its groups are whole vectors. The grid is a multiple of 8 (or
// one CTA per row), so that boundary is at the same column for every row of a CTA.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "host_common.h"
#include "ptx.cuh"
#include "schedule.h"

namespace dtcp {

constexpr int kNormMaxCols = 32768 - 8;  // 4 groups of 8 columns x 1024 threads, less one group for the boundary

struct NormParams {
  const uint16_t* x;
  const uint16_t* r;  // or null
  const uint16_t* w;  // or null: all ones
  uint16_t* s;        // or null
  void* y;
  void* scales;
  float* rstd;  // or null
  long long ldx, ldr, lds, ldy;
  int rows, cols;
  float eps;
};

struct NormBackwardParams {
  const uint16_t* dy;
  const uint16_t* s;
  const uint16_t* w;
  const float* rstd;
  const uint16_t* ds;  // or null
  uint16_t* dx;
  float* partial;  // [grid][cols], or null
  long long lddy, lds, ldds, lddx;
  int rows, cols;
};

namespace {

__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return pack_bf16x2_rn(__float_as_uint(lo), __float_as_uint(hi));
}

struct F8 {
  float v[8];
};
__device__ __forceinline__ F8 unpack8(uint4 p) {
  return F8{{bf_lo(p.x), bf_hi(p.x), bf_lo(p.y), bf_hi(p.y), bf_lo(p.z), bf_hi(p.z), bf_lo(p.w), bf_hi(p.w)}};
}
__device__ __forceinline__ uint4 pack8(const F8& f) {
  return make_uint4(pack2(f.v[0], f.v[1]), pack2(f.v[2], f.v[3]), pack2(f.v[4], f.v[5]), pack2(f.v[6], f.v[7]));
}

// Columns c .. c+7 of a row as BF16, zero outside [0, cols). ALIGNED: c and cols are multiples
// of 8 and the row starts on a 16-byte boundary.
template <bool ALIGNED>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int cols) {
  if (ALIGNED) return c < cols ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
  if (c >= 0 && c + 8 <= cols && (reinterpret_cast<uintptr_t>(row + c) & 15u) == 0)
    return *reinterpret_cast<const uint4*>(row + c);
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = (c + j >= 0 && c + j < cols) ? row[c + j] : 0u;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

template <bool ALIGNED>
__device__ __forceinline__ void store8(uint16_t* row, int c, int cols, uint4 v) {
  if (ALIGNED) {
    if (c < cols) *reinterpret_cast<uint4*>(row + c) = v;
    return;
  }
  if (c >= 0 && c + 8 <= cols && (reinterpret_cast<uintptr_t>(row + c) & 15u) == 0) {
    *reinterpret_cast<uint4*>(row + c) = v;
    return;
  }
  const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= 0 && c + j < cols) row[c + j] = static_cast<uint16_t>(e[j / 2] >> (16 * (j & 1)));
}

template <bool ALIGNED>
__device__ __forceinline__ void store8_bytes(uint8_t* row, int c, int cols, uint2 v) {
  if (c >= 0 && c + 8 <= cols && (ALIGNED || (reinterpret_cast<uintptr_t>(row + c) & 7u) == 0)) {
    *reinterpret_cast<uint2*>(row + c) = v;
    return;
  }
  if (ALIGNED) return;
  const uint32_t e[2] = {v.x, v.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= 0 && c + j < cols) row[c + j] = static_cast<uint8_t>(e[j / 4] >> (8 * (j & 3)));
}

// Four FP32 values -> E4M3 codes (to nearest, ties to even; beyond 448 -> 448; NaN -> NaN), first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

// One FP32 value -> E4M3 code, and the value of the code.
__device__ __forceinline__ uint32_t e4m3_code(float v) { return e4m3x4(v, 0.0f, 0.0f, 0.0f) & 0xFFu; }
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;  // two FP16 values
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(static_cast<uint16_t>(h & 0xFFFFu)));
  return f;
}

// Eight FP32 values -> E2M1 codes (to nearest, ties to even; beyond 6 -> 6), first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the CTA, the same bits in every thread. `slots` (one float per warp) is free again
// after the next CTA-wide barrier, so callers alternate between buffers.
__device__ __forceinline__ float block_sum(float v, float* slots, int warps) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : 0.0f);
}

// The largest of non-negative floats given as bits (NaN counts as larger than infinity).
__device__ __forceinline__ uint32_t block_max_bits(uint32_t v, uint32_t* slots, int warps) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : 0u);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The columns by which a row starts past a 16-byte boundary.
__device__ __forceinline__ int row_phase(const uint16_t* row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(row) >> 1) & 7u);
}

// ---------------------------------------------------------------- forward

template <int VPT, int FORMAT, bool ALIGNED>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
  __shared__ float slots[2][32];
  __shared__ uint32_t slots_max[2][32];
  const int warps = blockDim.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int phase = ALIGNED ? 0 : row_phase(p.x + blockIdx.x * p.ldx);
  int col[VPT];
  uint4 w[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    col[k] = 8 * (static_cast<int>(threadIdx.x) + k * static_cast<int>(blockDim.x)) - phase;
    constexpr uint32_t kOnes = 0x3F803F80u;
    w[k] = p.w != nullptr ? load8<ALIGNED>(p.w, col[k], p.cols) : make_uint4(kOnes, kOnes, kOnes, kOnes);
  }
  int parity = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    uint4 s[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) s[k] = load8<ALIGNED>(p.x + row * p.ldx, col[k], p.cols);
    if (p.r != nullptr) {
      uint4 r[VPT];
#pragma unroll
      for (int k = 0; k < VPT; ++k) r[k] = load8<ALIGNED>(p.r + row * p.ldr, col[k], p.cols);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        F8 a = unpack8(s[k]);
        const F8 b = unpack8(r[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] += b.v[j];
        s[k] = pack8(a);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (p.s != nullptr) store8<ALIGNED>(p.s + row * p.lds, col[k], p.cols, s[k]);
      const F8 a = unpack8(s[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(a.v[j], a.v[j], sum);
    }
    sum = block_sum(sum, slots[parity], warps);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(p.cols) + p.eps);
    if (p.rstd != nullptr && threadIdx.x == 0) p.rstd[row] = rstd;
    if constexpr (FORMAT == GEMM_NORM_BF16) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        F8 a = unpack8(s[k]);
        const F8 g = unpack8(w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] = a.v[j] * rstd * g.v[j];
        store8<ALIGNED>(static_cast<uint16_t*>(p.y) + row * p.ldy, col[k], p.cols, pack8(a));
      }
    } else if constexpr (FORMAT == GEMM_NORM_E4M3) {
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const F8 a = unpack8(s[k]), g = unpack8(w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (ALIGNED || (col[k] + j >= 0 && col[k] + j < p.cols)) top = max(top, abs_bits(a.v[j] * rstd * g.v[j]));
      }
      top = block_max_bits(top, slots_max[parity], warps);
      const float scale = __uint_as_float(top) / 448.0f;
      // (finite for a row of denormals too; a NaN stays one)
      float inverse = top == 0 ? 0.0f : 448.0f / __uint_as_float(top);
      if (inverse > 3.0e38f) inverse = 3.0e38f;
      if (threadIdx.x == 0) static_cast<float*>(p.scales)[row] = scale;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        F8 a = unpack8(s[k]);
        const F8 g = unpack8(w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] = a.v[j] * rstd * g.v[j] * inverse;
        store8_bytes<ALIGNED>(static_cast<uint8_t*>(p.y) + row * p.ldy, col[k], p.cols,
                              make_uint2(e4m3x4(a.v[0], a.v[1], a.v[2], a.v[3]), e4m3x4(a.v[4], a.v[5], a.v[6], a.v[7])));
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        F8 a = unpack8(s[k]);
        const F8 g = unpack8(w[k]);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a.v[j] = a.v[j] * rstd * g.v[j];
          top = max(top, abs_bits(a.v[j]));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the other 8 of the block's 16 columns
        const uint32_t code = e4m3_code(__uint_as_float(top) / 6.0f);
        const float sf = e4m3_value(code);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] = sf > 0.0f ? a.v[j] / sf : 0.0f;
        if (col[k] < p.cols) {
          static_cast<uint32_t*>(p.y)[(row * p.cols + col[k]) / 8] = e2m1x8(a.v);
          if ((threadIdx.x & 1) == 0)
            static_cast<uint8_t*>(p.scales)[(row * p.cols + col[k]) / 16] = static_cast<uint8_t>(code);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- backward

template <int VPT, bool ALIGNED>
__global__ void __launch_bounds__(1024) rms_norm_backward_kernel(const NormBackwardParams p) {
  __shared__ float slots[2][32];
  const int warps = blockDim.x >> 5;
  pdl_launch_dependents();
  pdl_wait();
  const int phase = ALIGNED ? 0 : row_phase(p.s + blockIdx.x * p.lds);
  int col[VPT];
  uint4 w[VPT];
  F8 dw[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    col[k] = 8 * (static_cast<int>(threadIdx.x) + k * static_cast<int>(blockDim.x)) - phase;
    constexpr uint32_t kOnes = 0x3F803F80u;
    w[k] = p.w != nullptr ? load8<ALIGNED>(p.w, col[k], p.cols) : make_uint4(kOnes, kOnes, kOnes, kOnes);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[k].v[j] = 0.0f;
  }
  int parity = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    uint4 s[VPT], dy[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      s[k] = load8<ALIGNED>(p.s + row * p.lds, col[k], p.cols);
      dy[k] = load8<ALIGNED>(p.dy + row * p.lddy, col[k], p.cols);
    }
    const float rstd = p.rstd[row];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const F8 a = unpack8(s[k]), d = unpack8(dy[k]), g = unpack8(w[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = a.v[j] * rstd;
        dw[k].v[j] = fmaf(d.v[j], xh, dw[k].v[j]);
        sum = fmaf(d.v[j] * g.v[j], xh, sum);
      }
    }
    const float c = block_sum(sum, slots[parity], warps) / static_cast<float>(p.cols);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const F8 a = unpack8(s[k]), d = unpack8(dy[k]), g = unpack8(w[k]);
      F8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = rstd * (d.v[j] * g.v[j] - a.v[j] * rstd * c);
      if (p.ds != nullptr) {
        const F8 e = unpack8(load8<ALIGNED>(p.ds + row * p.ldds, col[k], p.cols));
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] += e.v[j];
      }
      store8<ALIGNED>(p.dx + row * p.lddx, col[k], p.cols, pack8(o));
    }
  }
  if (p.partial != nullptr) {
    float* out = p.partial + static_cast<long long>(blockIdx.x) * p.cols;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col[k] + j >= 0 && col[k] + j < p.cols) out[col[k] + j] = dw[k].v[j];
  }
}

// dw[c] = sum of the partial rows in order: 8 warps take every eighth row of 32 columns, then add up.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* partial, int rows, int cols, float* dw) {
  __shared__ float part[8][33];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < cols)
    for (int r = warp; r < rows; r += 8) v += partial[static_cast<long long>(r) * cols + c];
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < cols) {
    v = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += part[k][lane];
    dw[c] = v;
  }
}

// ---------------------------------------------------------------- host side

struct NormShape {
  int threads, vpt, grid;
};

// Threads and groups per thread that hold a row, and persistent CTAs to fill the SMs' threads.
NormShape norm_shape(int rows, int cols, int num_sms, bool aligned) {
  const int groups = ceil_div(cols, 8) + (aligned ? 0 : 1);
  NormShape s;
  s.vpt = groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4;
  s.threads = std::max(32, ceil_div(ceil_div(groups, s.vpt), 32) * 32);
  const int per_sm = std::max(1, 2048 / s.threads);
  const int most = std::max(8, num_sms * std::min(per_sm, 8) / 8 * 8);
  s.grid = std::min(rows, most);
  return s;
}

template <typename P, typename K>
int launch(K kernel, int grid, int threads, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

template <int FORMAT>
int launch_forward(const NormShape& s, bool aligned, cudaStream_t stream, const NormParams& p) {
  if (aligned) {
    if (s.vpt == 1) return launch(rms_norm_kernel<1, FORMAT, true>, s.grid, s.threads, stream, p);
    if (s.vpt == 2) return launch(rms_norm_kernel<2, FORMAT, true>, s.grid, s.threads, stream, p);
    return launch(rms_norm_kernel<4, FORMAT, true>, s.grid, s.threads, stream, p);
  }
  if constexpr (FORMAT != GEMM_NORM_NVFP4) {
    if (s.vpt == 1) return launch(rms_norm_kernel<1, FORMAT, false>, s.grid, s.threads, stream, p);
    if (s.vpt == 2) return launch(rms_norm_kernel<2, FORMAT, false>, s.grid, s.threads, stream, p);
    return launch(rms_norm_kernel<4, FORMAT, false>, s.grid, s.threads, stream, p);
  }
  return GEMM_ERR_MISALIGNED;
}

// Whether every row of a tensor of 2-byte elements starts on a 16-byte boundary.
bool rows_aligned(const void* p, long long ld, int bytes = 16) {
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && ld % 8 == 0;
}
bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_rms_norm(const void* X, const void* R, const void* W, void* S, void* Y, void* scales, float* rstd, int rows,
                  int cols, float eps, int format, void* stream, const gemm_norm_strides_t* strides) {
  if (rows < 0 || cols < 0 || !(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  if (format != GEMM_NORM_BF16 && format != GEMM_NORM_E4M3 && format != GEMM_NORM_NVFP4) return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_OK;
  if (X == nullptr || Y == nullptr || (format != GEMM_NORM_BF16 && scales == nullptr)) return GEMM_ERR_INVALID_ARG;
  if (R != nullptr && S == nullptr) return GEMM_ERR_INVALID_ARG;
  NormParams p;
  p.ldx = p.ldr = p.lds = p.ldy = cols;
  if (strides != nullptr) {
    if (strides->x) p.ldx = strides->x;
    if (strides->residual) p.ldr = strides->residual;
    if (strides->sum) p.lds = strides->sum;
    if (strides->y) p.ldy = strides->y;
    if (p.ldx < cols || p.ldr < cols || p.lds < cols || p.ldy < cols) return GEMM_ERR_INVALID_ARG;
  }
  if (cols > kNormMaxCols || (format == GEMM_NORM_NVFP4 && (cols % 16 != 0 || p.ldy != cols)))
    return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (misaligned(X, 2) || misaligned(R, 2) || misaligned(W, 2) || misaligned(S, 2) || misaligned(rstd, 4) ||
      misaligned(Y, format == GEMM_NORM_BF16 ? 2 : format == GEMM_NORM_E4M3 ? 1 : 4) ||
      misaligned(scales, format == GEMM_NORM_E4M3 ? 4 : 1))
    return GEMM_ERR_MISALIGNED;
  p.x = static_cast<const uint16_t*>(X);
  p.r = static_cast<const uint16_t*>(R);
  p.w = static_cast<const uint16_t*>(W);
  p.s = static_cast<uint16_t*>(S);
  p.y = Y;
  p.scales = scales;
  p.rstd = rstd;
  p.rows = rows;
  p.cols = cols;
  p.eps = eps;
  const bool aligned = cols % 8 == 0 && rows_aligned(X, p.ldx) && (R == nullptr || rows_aligned(R, p.ldr)) &&
                       rows_aligned(W, 0) && (S == nullptr || rows_aligned(S, p.lds)) &&
                       (format == GEMM_NORM_NVFP4 || rows_aligned(Y, p.ldy, format == GEMM_NORM_BF16 ? 16 : 8));
  if (format == GEMM_NORM_NVFP4 && !aligned) return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  const NormShape shape = norm_shape(rows, cols, info->num_sms, aligned);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (format == GEMM_NORM_BF16) return launch_forward<GEMM_NORM_BF16>(shape, aligned, s, p);
  if (format == GEMM_NORM_E4M3) return launch_forward<GEMM_NORM_E4M3>(shape, aligned, s, p);
  return launch_forward<GEMM_NORM_NVFP4>(shape, aligned, s, p);
}

int gemm_rms_norm_backward(const void* dY, const void* S, const void* W, const float* rstd, const void* dS, void* dX,
                           float* dW, int rows, int cols, void* stream, const gemm_norm_backward_strides_t* strides) {
  if (rows < 0 || cols < 0) return GEMM_ERR_INVALID_ARG;
  if (cols == 0) return GEMM_OK;
  if (rows > 0 && (dY == nullptr || S == nullptr || rstd == nullptr || dX == nullptr)) return GEMM_ERR_INVALID_ARG;
  NormBackwardParams p;
  p.lddy = p.lds = p.ldds = p.lddx = cols;
  if (strides != nullptr) {
    if (strides->dy) p.lddy = strides->dy;
    if (strides->sum) p.lds = strides->sum;
    if (strides->dsum) p.ldds = strides->dsum;
    if (strides->dx) p.lddx = strides->dx;
    if (p.lddy < cols || p.lds < cols || p.ldds < cols || p.lddx < cols) return GEMM_ERR_INVALID_ARG;
  }
  if (cols > kNormMaxCols) return GEMM_ERR_UNSUPPORTED_SHAPE;
  if (misaligned(dY, 2) || misaligned(S, 2) || misaligned(W, 2) || misaligned(rstd, 4) || misaligned(dS, 2) ||
      misaligned(dX, 2) || misaligned(dW, 4))
    return GEMM_ERR_MISALIGNED;
  if (rows == 0 && dW == nullptr) return GEMM_OK;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {  // the sum over no rows
    if (cudaMemsetAsync(dW, 0, static_cast<size_t>(cols) * 4, st) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
  }
  p.dy = static_cast<const uint16_t*>(dY);
  p.s = static_cast<const uint16_t*>(S);
  p.w = static_cast<const uint16_t*>(W);
  p.rstd = rstd;
  p.ds = static_cast<const uint16_t*>(dS);
  p.dx = static_cast<uint16_t*>(dX);
  p.partial = nullptr;
  p.rows = rows;
  p.cols = cols;
  const bool aligned = cols % 8 == 0 && rows_aligned(dY, p.lddy) && rows_aligned(S, p.lds) && rows_aligned(W, 0) &&
                       (dS == nullptr || rows_aligned(dS, p.ldds)) && rows_aligned(dX, p.lddx);
  const NormShape shape = norm_shape(rows, cols, info->num_sms, aligned);
  void* ws = nullptr;
  if (dW != nullptr && shape.grid > 1) {
    cudaMemPool_t pool = workspace_pool(device);
    if (pool == nullptr ||
        cudaMallocFromPoolAsync(&ws, static_cast<size_t>(shape.grid) * cols * 4, pool, st) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_OUT_OF_MEMORY;
    }
    p.partial = static_cast<float*>(ws);
  } else if (dW != nullptr) {
    p.partial = dW;  // one CTA: its partial row is the sum
  }
  int rc;
  if (aligned)
    rc = shape.vpt == 1   ? launch(rms_norm_backward_kernel<1, true>, shape.grid, shape.threads, st, p)
         : shape.vpt == 2 ? launch(rms_norm_backward_kernel<2, true>, shape.grid, shape.threads, st, p)
                          : launch(rms_norm_backward_kernel<4, true>, shape.grid, shape.threads, st, p);
  else
    rc = shape.vpt == 1   ? launch(rms_norm_backward_kernel<1, false>, shape.grid, shape.threads, st, p)
         : shape.vpt == 2 ? launch(rms_norm_backward_kernel<2, false>, shape.grid, shape.threads, st, p)
                          : launch(rms_norm_backward_kernel<4, false>, shape.grid, shape.threads, st, p);
  if (ws != nullptr) {
    if (rc == GEMM_OK) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(cols, 32)), 1, 1);
      cfg.blockDim = dim3(256, 1, 1);
      cfg.stream = st;
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaLaunchKernelEx(&cfg, column_sum_kernel, static_cast<const float*>(p.partial), shape.grid, cols, dW) !=
          cudaSuccess) {
        cudaGetLastError();
        rc = GEMM_ERR_LAUNCH;
      } else {
        count_launch();
      }
    }
    if (cudaFreeAsync(ws, st) != cudaSuccess && rc == GEMM_OK) rc = GEMM_ERR_LAUNCH;
  }
  return rc;
}

}  // extern "C"
