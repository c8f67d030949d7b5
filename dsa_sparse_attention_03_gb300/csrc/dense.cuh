// Launcher of the dense attention kernels (dense.cu), used by api.cu.
#pragma once

#include "common.cuh"
#include "dsa_dense.h"

namespace dsa {

// How a problem is cut: row tiles of 128 packed rows per CTA (nw), CTAs along
// the rows (tiles, an upper bound) and parts of the positions (splits).
struct DenseShape {
  int nw, tiles, splits;
};
DenseShape dense_shape(const dsa_dense_problem& p);

// part [R * H_q, splits, D_v] and ml [R * H_q, splits, 2] are used with splits > 1.
cudaError_t launch_dense(const dsa_dense_problem& p, const DenseShape& s, uint16_t* out, float* lse, float* part,
                         float* ml, uint32_t* status, cudaStream_t st);

}  // namespace dsa
