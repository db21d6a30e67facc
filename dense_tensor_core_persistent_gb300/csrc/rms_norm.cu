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

#include "norm_common.cuh"

namespace dtcp {

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

// ---------------------------------------------------------------- forward

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
    auto value = [&](int k) {
      F8 a = unpack8(s[k]);
      const F8 g = unpack8(w[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) a.v[j] = a.v[j] * rstd * g.v[j];
      return a;
    };
    norm_output<VPT, FORMAT, ACCESS>(value, p.y, p.ldy, p.scales, row, p.cols, col, slots_max[parity], warps);
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
