// loss_common.cuh -- what the cross entropy's kernels share: partial softmax statistics, and the few-row kernel's launch.
#pragma once

#include "common.cuh"
#include "host_common.h"

namespace dtcp {

constexpr float kLog2e = 1.4426950408889634f;

// scale / ln 2; finite, so that equal logits stay apart by nothing.
__device__ __forceinline__ float log2_scale(float scale) { return fminf(scale * kLog2e, 3.4028234663852886e38f); }

// The maximum of a set of logits and the sum of exp(scale (z - m)) over all of them but one that is the maximum.
struct SoftmaxPart {
  float m, others;
};
__device__ __forceinline__ SoftmaxPart join(SoftmaxPart a, SoftmaxPart b, float c) {  // c = scale / ln 2
  if (b.m > a.m) {
    const SoftmaxPart t = a;
    a = b;
    b = t;
  }
  // (equal maxima, both minus infinity among them, count 1; a NaN among the others stays one)
  const float w = a.m == b.m ? 1.0f : ex2_approx((b.m - a.m) * c);
  return SoftmaxPart{a.m, fmaf(b.others + 1.0f, w, a.others)};
}

// What a row's logits become in the gradient: scale ((dloss + dlse) p - dloss 1[target]).
struct LossGradient {
  const long long* targets;  // or null
  const float* lse;
  const float* dloss;  // or null
  const float* dlse;   // or null
  int rows, vocab, first_col;  // the piece's first column
  float scale;
};
struct GradientRow {
  float lse, softmax, onehot;
  bool dead;         // no gradient reaches the row: G is 0 whatever its logits are
  long long target;  // among the piece's columns
  __device__ __forceinline__ GradientRow() {}
  __device__ __forceinline__ GradientRow(const LossGradient& p, int row) {
    target = -1;
    lse = softmax = onehot = 0.0f;
    if (row < p.rows) {
      const long long t = p.targets != nullptr ? p.targets[row] : -1;
      lse = p.lse[row];
      if (t >= 0 && p.dloss != nullptr) {
        onehot = t < p.vocab ? p.dloss[row] : __int_as_float(0x7FC00000);
        target = t - p.first_col;
      }
      softmax = onehot + (p.dlse != nullptr ? p.dlse[row] : 0.0f);
    }
    dead = onehot == 0.0f && softmax == 0.0f;
    softmax *= p.scale;
    onehot *= p.scale;
  }
};
// Without the target's share.
__device__ __forceinline__ float gradient_of(float z, float scale, float lse, float softmax, bool dead) {
  const float e = ex2_approx(fmaf(z, scale, -lse) * kLog2e) * softmax;
  return dead ? 0.0f : e;
}

// Up to 64 rows of X against all of W (cross_entropy_rows.cu): parts receives [CTAs][rows], target_z a logit for each row
// with a target. Measured on GB300 against the pair tile: see there.
constexpr int kLossRows = 64;
struct LossRowsOperands {
  const void* x;
  const void* w;
  const long long* targets;  // or null
  float2* parts;
  float* target_z;
  long long ldx;
  int rows, vocab, depth;
  float scale;
};
// CTAs of the launch (and so parts of a row).
int loss_rows_ctas(int vocab, const DeviceInfo* info);
int run_loss_rows(const LossRowsOperands& p, int device, const DeviceInfo* info, cudaStream_t stream);
// The same for the gradient: G of the piece of `vocab` columns whose rows of W start at w, as the sum of two BF16 numbers:
// 2 * rows rows, ldg apart, the second half what the first one's rounding left. x_twice (or null) receives X's rows twice,
// ldx_twice apart, for the product with both halves.
struct LossRowsGradient {
  LossGradient row;
  uint16_t* g;
  long long ldg;
  uint16_t* x_twice;
  long long ldx_twice;
};
int run_loss_rows_gradient(const LossRowsOperands& p, const LossRowsGradient& grad, int device, const DeviceInfo* info,
                           cudaStream_t stream);

}  // namespace dtcp
