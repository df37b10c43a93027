// Internal interface between the block-scaled products' host code (block_host.cu)
// and the pair kernels' unit (block_pair.cu).
#pragma once

#include "block_few.cuh"
#include "host.h"

namespace dgt {

struct BlockLaunch {
  CUtensorMap tmP, tmQ;  // row and column operand
  CUtensorMap tmC;       // valid when p.g.c_tma
  BlockParams p;
  int grid;  // CTAs
  int dev;
  cudaStream_t stream;
};

// bn: 256 or 128 columns a tile; cols: a scale for each row of the column operand.
cudaError_t launch_block_pair(const BlockLaunch& L, int bn, bool cols);

}  // namespace dgt
