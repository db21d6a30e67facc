// glu_common.cuh -- what the gated feed-forward block's two tiles share.
#pragma once

#include "pair_tile.cuh"

namespace dtcp {

struct GluParams : PairParams {
  int act, save;
  const float* x_scale;  // E4M3: scales of X's rows, Wg's and Wu's
  const float* g_scale;
  const float* u_scale;
};

// The 512 x 256 pair tile (glu_wide.cu): p's product is planned for it, `clusters` pairs take it.
int glu_wide_max_clusters(int device);
int glu_wide_launch(const PairMaps& m, const GluParams& p, int clusters, cudaStream_t stream);

}  // namespace dtcp
