// norm_common.cuh -- what the row norms share: how a thread holds its groups of 8 columns of a row, fetches the next row
// ahead and stores its results, conversions to 8 and 4 bits, sums over a CTA, and the shapes of the launches. Both norms
// are bound by the bytes they move; rms_norm.cu says why rows are held and fetched this way.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host_common.h"
#include "ptx.cuh"
#include "schedule.h"

namespace dtcp {

// Dynamic shared memory of a CTA, at most: three inputs of two rows and a weight, four groups a thread.
constexpr int kNormMaxSmem = (2 * 3 + 1) * 4 * 512 * 16;
constexpr float kNormMostInverse = 1.7014118346046923e38f;  // 2^127, of an E4M3 row's scale
constexpr int kNormMaxCols = 32768 - 8;  // 8 groups of 8 columns x 512 threads, less one group for the boundary

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

// Eight values as four packed pairs.
struct P8 {
  uint64_t v[4];
};
__device__ __forceinline__ P8 unpack8_pairs(uint4 p) {
  return P8{{f2_pack(bf_lo(p.x), bf_hi(p.x)), f2_pack(bf_lo(p.y), bf_hi(p.y)), f2_pack(bf_lo(p.z), bf_hi(p.z)),
             f2_pack(bf_lo(p.w), bf_hi(p.w))}};
}

// How the rows of a call's tensors lie against the groups of 8 columns.
enum NormAccess {
  kAligned = 0,  // every row starts on a 16-byte boundary, cols a multiple of 8
  kShared = 1,   // all tensors share their misalignment: whole vectors but in a row's first and last group
  kElements = 2  // anything else: element by element
};

__device__ __forceinline__ bool whole(int c, int cols) { return c >= 0 && c + 8 <= cols; }
__device__ __forceinline__ bool edge(int c, int cols) { return !whole(c, cols) && c + 8 > 0 && c < cols; }

__device__ __forceinline__ uint4 load_elements(const uint16_t* row, int c, int cols) {
  uint32_t e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) e[j] = (c + j >= 0 && c + j < cols) ? row[c + j] : 0u;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// A thread's groups of NT rows (a null row is not read) on their way to its own places in shared memory: the copies run
// through the reduction and the stores of the row before, hold no registers, and put zeros for what lies past the row's
// end. Groups that start past it are not written. Whole vectors are read at a row's start too, and what lies before it
// is masked off later (mask_start), but for the first row, where it may lie before the tensor.
template <int NT, int VPT, int ACCESS>
__device__ __forceinline__ void fetch_rows(uint4* mine, const uint16_t* const (&row)[NT], const int (&col)[VPT],
                                           int cols, long long index) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (row[t] == nullptr) continue;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      uint4* at = mine + (t * VPT + k) * static_cast<int>(blockDim.x);
      if (ACCESS == kElements || (ACCESS == kShared && k == 0 && col[0] < 0 && index * cols < 7)) {
        *at = load_elements(row[t], col[k], cols);
      } else if (ACCESS == kAligned ? col[k] < cols : col[k] + 8 <= cols) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(at)), "l"(row[t] + col[k]) : "memory");
      } else if (ACCESS == kShared && col[k] < cols) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(at)), "l"(row[t] + col[k]),
                     "r"(2 * (cols - col[k]))
                     : "memory");
      }
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// What of a thread's first group (columns c ..) lies before the row becomes zero.
__device__ __forceinline__ void mask_start(uint4& v, int c) {
  v.x &= c >= 0 ? 0xFFFFFFFFu : c == -1 ? 0xFFFF0000u : 0u;
  v.y &= c >= -2 ? 0xFFFFFFFFu : c == -3 ? 0xFFFF0000u : 0u;
  v.z &= c >= -4 ? 0xFFFFFFFFu : c == -5 ? 0xFFFF0000u : 0u;
  v.w &= c >= -6 ? 0xFFFFFFFFu : c == -7 ? 0xFFFF0000u : 0u;
}

// Waits for the row fetched before the last one (SLOTS == 2), or for the last one.
template <int SLOTS>
__device__ __forceinline__ void wait_fetched() {
  if (SLOTS == 2)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Rows in shared memory at a time: eight groups leave room for one, and with one group a CTA has one row.
__host__ __device__ constexpr int norm_slots(int vpt) { return vpt == 2 || vpt == 4 ? 2 : 1; }

// The part of a vector of eight 2-byte elements that lies in the row, in at most three naturally aligned pieces a
// side (the vector's own place is 16-byte aligned): elements a .. b-1.
__device__ __forceinline__ void store_part(uint16_t* at, uint4 v, int a, int b) {
  if (a <= 0 && b >= 8) return;
  auto half = [&](int j) {
    const uint32_t w = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
    return static_cast<uint16_t>(j & 1 ? w >> 16 : w);
  };
  if (a > 0 && b >= 8) {  // a row's first group: the elements from a on
    if (a & 1) at[a] = half(a);
    const int c = (a + 1) & ~1;
    if (c & 2) *reinterpret_cast<uint32_t*>(at + c) = c == 2 ? v.y : v.w;
    if (c <= 4) *reinterpret_cast<uint2*>(at + 4) = make_uint2(v.z, v.w);
    return;
  }
  if (a <= 0) {  // its last group: the elements before b
    if (b & 4) *reinterpret_cast<uint2*>(at) = make_uint2(v.x, v.y);
    const int c = b & 4;
    if (b & 2) *reinterpret_cast<uint32_t*>(at + c) = c ? v.z : v.x;
    if (b & 1) at[b - 1] = half(b - 1);
    return;
  }
  for (int j = a; j < b; ++j) at[j] = half(j);  // a row inside one group
}

template <int ACCESS>
__device__ __forceinline__ void store8(uint16_t* row, int c, int cols, uint4 v) {
  if (ACCESS != kElements && (ACCESS == kAligned ? c < cols : whole(c, cols))) {
    *reinterpret_cast<uint4*>(row + c) = v;
    return;
  }
  if (ACCESS == kAligned) return;
  if (ACCESS == kShared) {
    if (edge(c, cols)) store_part(row + c, v, -c, cols - c);
    return;
  }
  const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= 0 && c + j < cols) row[c + j] = static_cast<uint16_t>(e[j / 2] >> (16 * (j & 1)));
}

template <int ACCESS>
__device__ __forceinline__ void store8_bytes(uint8_t* row, int c, int cols, uint2 v) {
  if (ACCESS != kElements && (ACCESS == kAligned ? c < cols : whole(c, cols))) {
    *reinterpret_cast<uint2*>(row + c) = v;
    return;
  }
  if (ACCESS == kAligned || (ACCESS == kShared && !edge(c, cols))) return;
  const uint32_t e[2] = {v.x, v.y};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= 0 && c + j < cols) row[c + j] = static_cast<uint8_t>(e[j / 4] >> (8 * (j & 3)));
}

// The weight of a thread's groups: once per CTA, so element by element unless rows are aligned.
template <int VPT, int ACCESS>
__device__ __forceinline__ void load_weight(uint4 (&w)[VPT], const uint16_t* weight, const int (&col)[VPT], int cols) {
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    constexpr uint32_t kOnes = 0x3F803F80u;
    w[k] = make_uint4(kOnes, kOnes, kOnes, kOnes);
    if (weight == nullptr) continue;
    if (ACCESS == kAligned)
      w[k] = col[k] < cols ? *reinterpret_cast<const uint4*>(weight + col[k]) : make_uint4(0u, 0u, 0u, 0u);
    else
      w[k] = load_elements(weight, col[k], cols);
  }
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

// An E4M3 row's scale and its inverse, from its largest magnitude's bits (a NaN stays one).
struct E4m3Scale {
  float scale, inverse;
  __device__ __forceinline__ explicit E4m3Scale(uint32_t top) {
    scale = __uint_as_float(top) / 448.0f;
    inverse = top == 0 ? 0.0f : 448.0f / __uint_as_float(top);
    if (inverse > kNormMostInverse) {  // a row near FP32's smallest numbers: the scale stops where its inverse does
      inverse = kNormMostInverse;
      scale = 1.0f / kNormMostInverse;
    }
  }
};

// A row's outputs in their format; value(k): the thread's eight results of group k, FP32.
template <int VPT, int FORMAT, int ACCESS, class Value>
__device__ __forceinline__ void norm_output(const Value& value, void* y, long long ldy, void* scales, long long row,
                                            int cols, const int (&col)[VPT], uint32_t* slots_max, int warps) {
  if constexpr (FORMAT == GEMM_NORM_BF16) {
#pragma unroll
    for (int k = 0; k < VPT; ++k)
      store8<ACCESS>(static_cast<uint16_t*>(y) + row * ldy, col[k], cols, pack8(value(k)));
  } else if constexpr (FORMAT == GEMM_NORM_E4M3) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const F8 a = value(k);
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, abs_bits(a.v[j]));
    }
    top = block_max_bits(top, slots_max, warps);
    const E4m3Scale s(top);
    if (threadIdx.x == 0) static_cast<float*>(scales)[row] = s.scale;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      F8 a = value(k);
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] *= s.inverse;
      store8_bytes<ACCESS>(static_cast<uint8_t*>(y) + row * ldy, col[k], cols,
                           make_uint2(e4m3x4(a.v[0], a.v[1], a.v[2], a.v[3]), e4m3x4(a.v[4], a.v[5], a.v[6], a.v[7])));
    }
  } else {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      F8 a = value(k);
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, abs_bits(a.v[j]));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));  // the other 8 of the block's 16 columns
      const uint32_t code = e4m3_code(__uint_as_float(top) / 6.0f);
      const float sf = e4m3_value(code);
      const float inverse = sf > 0.0f ? 1.0f / sf : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] *= inverse;
      if (col[k] < cols) {
        static_cast<uint32_t*>(y)[(row * cols + col[k]) / 8] = e2m1x8(a.v);
        if ((threadIdx.x & 1) == 0)
          static_cast<uint8_t*>(scales)[(row * cols + col[k]) / 16] = static_cast<uint8_t>(code);
      }
    }
  }
}

// Registers per thread by groups per thread: 1024 threads with one group, 512 with more. With two groups as few as
// hold a row without spills, so that several CTAs fit on an SM; with four a little fewer (4 to 36 bytes a thread are
// spilled in the gradient and in the RMS norm's rows to E4M3 off the boundary); with eight the 128 that 512 threads leave, which
// do not hold a row (RMS norm 44 to 76 bytes forward and 132 to 312 in the gradient, layer norm, whose values are FP32, 412 to
// 824 and 904 to 1760). Rows off the boundary need some more for their ends; measured on GB300 at 16000 x
// 1023: forward 25.1 us with 64 and 26.7 with 56, gradient 36.3 with 80 and 42.8 with 64.
template <int VPT>
constexpr int norm_regs(int two, int four) { return VPT == 1 ? 64 : VPT == 2 ? two : VPT == 4 ? four : 128; }

// ---------------------------------------------------------------- host side

// Groups of 8 columns per thread for many rows; measured on GB300: forward 4000 x 4096 17.9 us with 2 and 18.4 with 4,
// off the 16-byte boundary 4001 x 4099 22.7 and 27.7; its gradient 29.5 and 38.9.
constexpr int kNormGroups = 2;

struct NormShape {
  int threads, vpt;
};

// Threads and groups per thread that hold a row.
//   Few rows (no more than SMs): one group per thread, the shortest time from load to output.
//   Many rows: kNormGroups per thread, more where 512 threads do not hold a row.
inline NormShape norm_shape(int rows, int cols, int num_sms, bool aligned) {
  const int groups = ceil_div(cols, 8) + (aligned ? 0 : 1);
  NormShape s;
  s.vpt = rows <= num_sms ? 1 : kNormGroups;
  for (;; s.vpt *= 2) {
    const int most = s.vpt == 1 ? 1024 : 512;
    s.threads = std::max(32, ceil_div(ceil_div(groups, s.vpt), 32) * 32);
    if (s.threads <= most) return s;
  }
}

// Bytes of a CTA's rows in shared memory, of `tensors` inputs.
inline int norm_smem(const NormShape& shape, int tensors) {
  return norm_slots(shape.vpt) * tensors * shape.vpt * shape.threads * 16;
}

// CTAs of a persistent launch: as many as fit on the SMs together, a multiple of 8, or one per row; 0 on an error.
inline int norm_grid(const void* kernel, int rows, int threads, int smem, int num_sms) {
  if (smem > 46 * 1024 &&  // (a CTA has 48 KB without asking, a little of it for the reductions)
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return std::min(rows, std::max(8, num_sms * resident_ctas(kernel, threads, smem) / 8 * 8));
}

inline int norm_launch(const void* kernel, dim3 grid, dim3 threads, int smem, cudaStream_t stream, void** args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  count_launch();
  return GEMM_OK;
}

// A tensor's rows against 16-byte boundaries: the elements of the first row and of the stride past one.
struct RowPlace {
  unsigned first, stride;
  RowPlace(const void* p, long long ld, int bytes)
      : first(static_cast<unsigned>(reinterpret_cast<uintptr_t>(p) / bytes % 8)),
        stride(static_cast<unsigned>(ld % 8)) {}
  bool operator==(const RowPlace& o) const { return first == o.first && stride == o.stride; }
  bool aligned() const { return first == 0 && stride == 0; }
};

inline bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Zeros, as the sum over nothing is (a null pointer: nothing to do).
inline int zero_floats(void* p, int n, cudaStream_t stream) {
  if (p != nullptr && cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 4, stream) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace dtcp
