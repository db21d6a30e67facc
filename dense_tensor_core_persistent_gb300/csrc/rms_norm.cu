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
// Both directions are bound by the bytes they move (forward at most 8 per element, backward 8), so a row is read once:
// a thread holds 2 groups of 8 columns (4 or 8 in rows longer than 8192 or 16384), up to 512 threads hold a row. CTAs
// are persistent, as many as fit on the SMs, and step over rows by the grid size. Each thread copies its groups of the
// CTA's next row to places of its own in shared memory (cp.async) before it takes the current one from there, so
// loads stay in flight through the reductions and stores without holding registers or meeting at barriers. (With eight
// groups there is room for one row: the next one is asked for once the current one has been read, the gradient's once
// it has been written, so little of it streams.) A thread always owns the same columns: the weight is read once per
// CTA and the weight's gradient is summed in registers, one partial row per CTA, which a second kernel adds in a fixed
// order (no atomics).
//
// Rows that no 16-byte vector divides: the groups of a row start at its 16-byte boundary, so
// all but the first and last of its groups are whole vectors. The grid is a multiple of 8 (or
// one CTA per row), so that boundary is at the same column for every row of a CTA.
//
// Measured on GB300 with inputs larger than L2, residual added: 4000 x 8192 44 us in BF16 (5.9 TB/s) and 37.6 to E4M3
// (6.1), 4001 x 4099 24 us in both; gradient 4000 x 8192 45 us (5.8), with the weight's 51; 4001 x 4099 28 (4.7) and
// 32. Off the boundary the rest goes to the row ends' parts and the warps that a row fills in part. Short rows are a
// CTA of a few warps each, with a barrier a row: the gradient of 16000 x 1024 takes 24 us, with the weight's 34 (floor
// 19.6), 131072 x 128 71 and 88 (floor 20.1). With the rows loaded to registers (and as many groups a thread as were
// best then) the first ones took 43, 37, 24, 55, 66, 33 and 39 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "host_common.h"
#include "ptx.cuh"
#include "schedule.h"

namespace dtcp {

constexpr int kNormMaxSmem = 3 * 8 * 512 * 16;  // dynamic shared memory of a CTA: three inputs, eight groups
constexpr float kNormMostInverse = 1.7014118346046923e38f;  // 2^127, of an E4M3 row's scale
constexpr int kNormMaxCols = 32768 - 8;  // 8 groups of 8 columns x 512 threads, less one group for the boundary

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

// ---------------------------------------------------------------- forward

// Registers per thread by groups per thread: 1024 threads with one group, 512 with more. With two groups as few as
// hold a row without spills, so that several CTAs fit on an SM; with four a little fewer (4 to 40 bytes a thread are
// spilled in the gradient and in forward rows off the boundary); with eight the 128 that 512 threads leave, which do
// not hold a row (44 to 184 bytes). Rows off the boundary need some more for their ends; measured on GB300 at 16000 x
// 1023: forward 25.1 us with 64 and 26.7 with 56, gradient 36.3 with 80 and 42.8 with 64.
template <int VPT>
constexpr int norm_regs(int two, int four) { return VPT == 1 ? 64 : VPT == 2 ? two : VPT == 4 ? four : 128; }

template <int VPT, int FORMAT, int ACCESS>
__global__ void __maxnreg__(norm_regs<VPT>(ACCESS == kAligned ? 56 : 64, 80)) rms_norm_kernel(const NormParams p) {
  constexpr int SLOTS = norm_slots(VPT);
  extern __shared__ uint4 fetched[];  // [SLOTS][2][VPT][threads]
  __shared__ float slots[2][32];
  __shared__ uint32_t slots_max[2][32];
  const int warps = blockDim.x >> 5;
  uint4* const mine = fetched + threadIdx.x;
  const int slot_size = 2 * VPT * static_cast<int>(blockDim.x);
  pdl_launch_dependents();
  pdl_wait();
  const int phase = ACCESS == kAligned ? 0 : row_phase(p.x + blockIdx.x * p.ldx);
  int col[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    col[k] = 8 * (static_cast<int>(threadIdx.x) + k * static_cast<int>(blockDim.x)) - phase;
  auto fetch = [&](long long row, int slot) {
    const uint16_t* const rows[2] = {p.x + row * p.ldx, p.r != nullptr ? p.r + row * p.ldr : nullptr};
    fetch_rows<2, VPT, ACCESS>(mine + slot * slot_size, rows, col, p.cols, row);
  };
  // (groups past the row's end stay zero)
  for (int i = 0; i < SLOTS * 2 * VPT; ++i) mine[i * static_cast<int>(blockDim.x)] = make_uint4(0u, 0u, 0u, 0u);
  fetch(blockIdx.x, 0);
  uint4 w[VPT];
  load_weight<VPT, ACCESS>(w, p.w, col, p.cols);
  const bool starts = threadIdx.x < 32 && phase != 0;  // the warp with the row's start
  int parity = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    const bool more = row + gridDim.x < p.rows;
    if (SLOTS == 2 && more) {
      fetch(row + gridDim.x, parity ^ 1);
      wait_fetched<2>();
    } else {
      wait_fetched<1>();
    }
    const uint4* const in = mine + (SLOTS == 2 ? parity * slot_size : 0);
    uint4 s[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      s[k] = in[k * static_cast<int>(blockDim.x)];
      if (p.r != nullptr) {
        F8 a = unpack8(s[k]);
        const F8 b = unpack8(in[(VPT + k) * static_cast<int>(blockDim.x)]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] += b.v[j];
        s[k] = pack8(a);
      }
    }
    if (ACCESS == kShared && starts) mask_start(s[0], col[0]);
    if (SLOTS == 1 && more) fetch(row + gridDim.x, 0);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (p.s != nullptr) store8<ACCESS>(p.s + row * p.lds, col[k], p.cols, s[k]);
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
        store8<ACCESS>(static_cast<uint16_t*>(p.y) + row * p.ldy, col[k], p.cols, pack8(a));
      }
    } else if constexpr (FORMAT == GEMM_NORM_E4M3) {
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const F8 a = unpack8(s[k]), g = unpack8(w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          top = max(top, abs_bits(a.v[j] * rstd * g.v[j]));
      }
      top = block_max_bits(top, slots_max[parity], warps);
      float scale = __uint_as_float(top) / 448.0f;
      // (a NaN stays one)
      float inverse = top == 0 ? 0.0f : 448.0f / __uint_as_float(top);
      if (inverse > kNormMostInverse) {  // a row near FP32's smallest numbers: the scale stops where its inverse does
        inverse = kNormMostInverse;
        scale = 1.0f / kNormMostInverse;
      }
      if (threadIdx.x == 0) static_cast<float*>(p.scales)[row] = scale;
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        F8 a = unpack8(s[k]);
        const F8 g = unpack8(w[k]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] = a.v[j] * rstd * g.v[j] * inverse;
        store8_bytes<ACCESS>(static_cast<uint8_t*>(p.y) + row * p.ldy, col[k], p.cols,
                              make_uint2(e4m3x4(a.v[0], a.v[1], a.v[2], a.v[3]),
                                         e4m3x4(a.v[4], a.v[5], a.v[6], a.v[7])));
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
        const float inverse = sf > 0.0f ? 1.0f / sf : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a.v[j] *= inverse;
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

template <int VPT, int ACCESS>
__global__ void __maxnreg__(norm_regs<VPT>(ACCESS == kAligned ? 64 : 80, 96))
    rms_norm_backward_kernel(const NormBackwardParams p) {
  constexpr int SLOTS = norm_slots(VPT);
  extern __shared__ uint4 fetched[];  // [SLOTS][3][VPT][threads]
  __shared__ float slots[2][32];
  const int warps = blockDim.x >> 5;
  uint4* const mine = fetched + threadIdx.x;
  const int slot_size = 3 * VPT * static_cast<int>(blockDim.x);
  pdl_launch_dependents();
  pdl_wait();
  const int phase = ACCESS == kAligned ? 0 : row_phase(p.s + blockIdx.x * p.lds);
  int col[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
    col[k] = 8 * (static_cast<int>(threadIdx.x) + k * static_cast<int>(blockDim.x)) - phase;
  auto fetch = [&](long long row, int slot) {
    const uint16_t* const rows[3] = {p.s + row * p.lds, p.dy + row * p.lddy,
                                     p.ds != nullptr ? p.ds + row * p.ldds : nullptr};
    fetch_rows<3, VPT, ACCESS>(mine + slot * slot_size, rows, col, p.cols, row);
  };
  // (groups past the row's end stay zero)
  for (int i = 0; i < SLOTS * 3 * VPT; ++i) mine[i * static_cast<int>(blockDim.x)] = make_uint4(0u, 0u, 0u, 0u);
  fetch(blockIdx.x, 0);
  uint4 w[VPT];
  P8 dw[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[k].v[j] = 0;
  load_weight<VPT, ACCESS>(w, p.w, col, p.cols);
  const bool starts = threadIdx.x < 32 && phase != 0;  // the warp with the row's start
  const float mean = 1.0f / static_cast<float>(p.cols);
  float rstd = p.rstd[blockIdx.x], rstd_next = 0.0f;
  int parity = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, parity ^= 1) {
    const bool more = row + gridDim.x < p.rows;
    if (more) rstd_next = p.rstd[row + gridDim.x];
    if (SLOTS == 2 && more) {
      fetch(row + gridDim.x, parity ^ 1);
      wait_fetched<2>();
    } else {
      wait_fetched<1>();
    }
    const uint4* const in = mine + (SLOTS == 2 ? parity * slot_size : 0);
    const uint64_t r2 = f2_pack(rstd, rstd);
    uint64_t sum2 = 0;
    float lo, hi;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      uint4 v[2] = {in[k * static_cast<int>(blockDim.x)], in[(VPT + k) * static_cast<int>(blockDim.x)]};
      if (ACCESS == kShared && k == 0 && starts) {
        mask_start(v[0], col[0]);
        mask_start(v[1], col[0]);
      }
      const P8 a = unpack8_pairs(v[0]), d = unpack8_pairs(v[1]), g = unpack8_pairs(w[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint64_t xh = f2_mul(a.v[j], r2);
        dw[k].v[j] = f2_fma(d.v[j], xh, dw[k].v[j]);
        sum2 = f2_fma(f2_mul(d.v[j], g.v[j]), xh, sum2);
      }
    }
    f2_unpack(sum2, lo, hi);
    const float c = block_sum(lo + hi, slots[parity], warps) * mean;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const F8 a = unpack8(in[k * static_cast<int>(blockDim.x)]);
      const F8 d = unpack8(in[(VPT + k) * static_cast<int>(blockDim.x)]), g = unpack8(w[k]);
      F8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) o.v[j] = rstd * (d.v[j] * g.v[j] - a.v[j] * rstd * c);
      if (p.ds != nullptr) {
        const F8 e = unpack8(in[(2 * VPT + k) * static_cast<int>(blockDim.x)]);
#pragma unroll
        for (int j = 0; j < 8; ++j) o.v[j] += e.v[j];
      }
      store8<ACCESS>(p.dx + row * p.lddx, col[k], p.cols, pack8(o));
    }
    if (SLOTS == 1 && more) fetch(row + gridDim.x, 0);
    rstd = rstd_next;
  }
  if (p.partial != nullptr) {  // through shared memory, so that a warp writes 32 columns side by side
    float* const sums = reinterpret_cast<float*>(fetched);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      ulonglong2* at = reinterpret_cast<ulonglong2*>(sums + col[k] + phase);
      at[0] = make_ulonglong2(dw[k].v[0], dw[k].v[1]);
      at[1] = make_ulonglong2(dw[k].v[2], dw[k].v[3]);
    }
    __syncthreads();
    float* out = p.partial + static_cast<long long>(blockIdx.x) * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += blockDim.x) out[c] = sums[c + phase];
  }
}

// dw[c] = sum of the partial rows in a fixed order: 32 warps take every 32nd row of 32 columns, then a column each.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
    column_sum_kernel(const float* partial, int rows, int cols, float* dw) {
  __shared__ float part[kSumWarps][33];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int r = warp; r < rows; r += kSumWarps) v += partial[static_cast<long long>(r) * cols + c];
  part[warp][lane] = v;
  __syncthreads();
  v = warp_sum(part[lane][warp]);  // one column a warp
  if (lane == 0 && blockIdx.x * 32 + warp < cols) dw[blockIdx.x * 32 + warp] = v;
}

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
NormShape norm_shape(int rows, int cols, int num_sms, bool aligned) {
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
int norm_smem(const NormShape& shape, int tensors) {
  return norm_slots(shape.vpt) * tensors * shape.vpt * shape.threads * 16;
}

// CTAs of a persistent launch: as many as fit on the SMs together, a multiple of 8, or one per row; 0 on an error.
int norm_grid(const void* kernel, int rows, int threads, int smem, int num_sms) {
  if (smem > 46 * 1024 &&  // (a CTA has 48 KB without asking, a little of it for the reductions)
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kNormMaxSmem) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return std::min(rows, std::max(8, num_sms * resident_ctas(kernel, threads, smem) / 8 * 8));
}

int norm_launch(const void* kernel, int grid, int threads, int smem, cudaStream_t stream, void** args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
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

template <int FORMAT, int ACCESS>
const void* forward_kernel(int vpt) {
  return vpt == 1   ? reinterpret_cast<const void*>(rms_norm_kernel<1, FORMAT, ACCESS>)
         : vpt == 2 ? reinterpret_cast<const void*>(rms_norm_kernel<2, FORMAT, ACCESS>)
         : vpt == 4 ? reinterpret_cast<const void*>(rms_norm_kernel<4, FORMAT, ACCESS>)
                    : reinterpret_cast<const void*>(rms_norm_kernel<8, FORMAT, ACCESS>);
}
template <int FORMAT>
const void* forward_kernel(int vpt, bool aligned, bool shared) {
  return aligned  ? forward_kernel<FORMAT, kAligned>(vpt)
         : shared ? forward_kernel<FORMAT, kShared>(vpt)
                  : forward_kernel<FORMAT, kElements>(vpt);
}

template <int ACCESS>
const void* backward_kernel(int vpt) {
  return vpt == 1   ? reinterpret_cast<const void*>(rms_norm_backward_kernel<1, ACCESS>)
         : vpt == 2 ? reinterpret_cast<const void*>(rms_norm_backward_kernel<2, ACCESS>)
         : vpt == 4 ? reinterpret_cast<const void*>(rms_norm_backward_kernel<4, ACCESS>)
                    : reinterpret_cast<const void*>(rms_norm_backward_kernel<8, ACCESS>);
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

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Zeros, as the sum over nothing is (a null pointer: nothing to do).
int zero_floats(void* p, int n, cudaStream_t stream) {
  if (p != nullptr && cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 4, stream) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_LAUNCH;
  }
  return GEMM_OK;
}

}  // namespace
}  // namespace dtcp

using namespace dtcp;

extern "C" {

int gemm_rms_norm(const void* X, const void* R, const void* W, void* S, void* Y, void* scales, float* rstd, int rows,
                  int cols, float eps, int format, void* stream, const gemm_norm_strides_t* strides) {
  if (rows < 0 || cols < 0 || !(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
  if (format != GEMM_NORM_BF16 && format != GEMM_NORM_E4M3 && format != GEMM_NORM_NVFP4) return GEMM_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_OK;
  if (cols == 0) {  // rows without columns: what is one number a row is 0
    void* row_scales = format == GEMM_NORM_E4M3 ? scales : nullptr;
    if (row_scales == nullptr && rstd == nullptr) return GEMM_OK;
    if (misaligned(row_scales, 4) || misaligned(rstd, 4)) return GEMM_ERR_MISALIGNED;
    int device = 0, err = 0;
    if (current_device_info(&device, &err) == nullptr) return err;
    const int st = zero_floats(row_scales, rows, static_cast<cudaStream_t>(stream));
    return st != GEMM_OK ? st : zero_floats(rstd, rows, static_cast<cudaStream_t>(stream));
  }
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
  const RowPlace place(X, p.ldx, 2);
  bool shared = (R == nullptr || RowPlace(R, p.ldr, 2) == place) && (S == nullptr || RowPlace(S, p.lds, 2) == place);
  if (format == GEMM_NORM_BF16) shared = shared && RowPlace(Y, p.ldy, 2) == place;
  if (format == GEMM_NORM_E4M3) shared = shared && RowPlace(Y, p.ldy, 1) == place;  // (8-byte vectors of codes)
  const bool aligned = shared && place.aligned() && cols % 8 == 0 && !misaligned(W, 16);
  if (format == GEMM_NORM_NVFP4 && !aligned) return GEMM_ERR_MISALIGNED;
  int device = 0, err = 0;
  const DeviceInfo* info = current_device_info(&device, &err);
  if (info == nullptr) return err;
  const NormShape shape = norm_shape(rows, cols, info->num_sms, aligned);
  const void* kernel = format == GEMM_NORM_NVFP4  ? forward_kernel<GEMM_NORM_NVFP4, kAligned>(shape.vpt)
                       : format == GEMM_NORM_E4M3 ? forward_kernel<GEMM_NORM_E4M3>(shape.vpt, aligned, shared)
                                                  : forward_kernel<GEMM_NORM_BF16>(shape.vpt, aligned, shared);
  void* args[] = {&p};
  const int smem = norm_smem(shape, 2);
  const int grid = norm_grid(kernel, rows, shape.threads, smem, info->num_sms);
  if (grid == 0) return GEMM_ERR_LAUNCH;
  return norm_launch(kernel, grid, shape.threads, smem, static_cast<cudaStream_t>(stream), args);
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
  if (rows == 0) return zero_floats(dW, cols, st);  // the sum over no rows
  p.dy = static_cast<const uint16_t*>(dY);
  p.s = static_cast<const uint16_t*>(S);
  p.w = static_cast<const uint16_t*>(W);
  p.rstd = rstd;
  p.ds = static_cast<const uint16_t*>(dS);
  p.dx = static_cast<uint16_t*>(dX);
  p.partial = nullptr;
  p.rows = rows;
  p.cols = cols;
  const RowPlace place(S, p.lds, 2);
  const bool shared = RowPlace(dY, p.lddy, 2) == place && (dS == nullptr || RowPlace(dS, p.ldds, 2) == place) &&
                      RowPlace(dX, p.lddx, 2) == place;
  const bool aligned = shared && place.aligned() && cols % 8 == 0 && !misaligned(W, 16);
  const NormShape shape = norm_shape(rows, cols, info->num_sms, aligned);
  const void* kernel = aligned  ? backward_kernel<kAligned>(shape.vpt)
                       : shared ? backward_kernel<kShared>(shape.vpt)
                                : backward_kernel<kElements>(shape.vpt);
  const int smem = norm_smem(shape, 3);
  const int grid = norm_grid(kernel, rows, shape.threads, smem, info->num_sms);
  if (grid == 0) return GEMM_ERR_LAUNCH;
  void* ws = nullptr;
  if (dW != nullptr && grid > 1) {
    cudaMemPool_t pool = workspace_pool(device);
    if (pool == nullptr ||
        cudaMallocFromPoolAsync(&ws, static_cast<size_t>(grid) * cols * 4, pool, st) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_OUT_OF_MEMORY;
    }
    p.partial = static_cast<float*>(ws);
  } else if (dW != nullptr) {
    p.partial = dW;  // one CTA: its partial row is the sum
  }
  void* args[] = {&p};
  int rc = norm_launch(kernel, grid, shape.threads, smem, st, args);
  if (ws != nullptr) {
    if (rc == GEMM_OK) {
      const float* partial = p.partial;
      int partial_rows = grid;
      void* sum_args[] = {&partial, &partial_rows, &cols, &dW};
      rc = norm_launch(reinterpret_cast<const void*>(column_sum_kernel), ceil_div(cols, 32), 32 * kSumWarps, 0, st,
                       sum_args);
    }
    if (cudaFreeAsync(ws, st) != cudaSuccess && rc == GEMM_OK) rc = GEMM_ERR_LAUNCH;
  }
  return rc;
}

}  // extern "C"
